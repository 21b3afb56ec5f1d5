"""The expert layer's definition in 64 bits (numpy), with the fp32 roundings
that the casts name.  Shares no code with the library."""
import numpy as np

from tests.fp4_reference import E4M3, _nearest


def cast(v):
    """float64 [..., K] -> the values of its E4M3 codes times their fp32
    scales, one per 128 consecutive values."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    s = (np.abs(b).max(axis=-1, keepdims=True) / 448.0).astype(np.float32).astype(np.float64)
    s[s == 0] = 1.0
    q = (b / s).astype(np.float32).astype(np.float64)
    return (np.sign(q) * E4M3[_nearest(np.abs(q), E4M3[:127])] * s).reshape(v.shape)


def route(x, wr, k, renorm):
    """(ids [M, k], weights [M, k], the least gap between a chosen logit and
    the next one down) from float64 inputs."""
    logits = x @ wr.T
    order = np.argsort(-logits, axis=1, kind="stable")
    top = np.take_along_axis(logits, order, axis=1)
    p = np.exp(top - top[:, :1])
    w = p[:, :k] / (p[:, :k] if renorm else p).sum(axis=1, keepdims=True)
    gaps = (top[:, :-1] - top[:, 1:])[:, :k]
    return order[:, :k], w, float(gaps.min()) if gaps.size else np.inf


def experts(x, ids, weights, w13, w2):
    """(y, bound) from float64 x [M, H], dequantised w13 [E, 2I, H] and w2 [E, H, I];
    bound = sum of |w| |h| |w2|, for the tolerance."""
    E, H, I = w2.shape
    a = cast(x)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for e in range(E):
        m, j = np.nonzero(ids == e)
        if not m.size:
            continue
        gu = a[m] @ w13[e].T
        g, u = gu[:, :I], gu[:, I:]
        h = cast(g / (1.0 + np.exp(-g)) * u)
        w = weights[m, j].astype(np.float64)[:, None]
        np.add.at(y, m, (h @ w2[e].T) * w)
        np.add.at(bound, m, (np.abs(h) @ np.abs(w2[e]).T) * np.abs(w))
    return y, bound


def weights(E, rows, K, rng, std=0.05):
    """Random E4M3 codes [E, rows, K] and block scales [E * rows/128, K/128]
    as a quantiser leaves them, and the values they stand for."""
    w = rng.standard_normal((E * rows // 128, 128, K // 128, 128)) * std
    s = (np.abs(w).max(axis=(1, 3)) / 448.0).astype(np.float32)
    q = w / s[:, None, :, None]
    mag = _nearest(np.abs(q), E4M3[:127])
    codes = (mag + 128 * ((q < 0) & (mag > 0))).astype(np.uint8)
    v = E4M3[codes] * s.astype(np.float64)[:, None, :, None]
    return codes.reshape(E, rows, K), s, v.reshape(E, rows, K)


def tile(codes):
    """Row-major codes [E, rows, K] -> the tiled layout [tiles, 128, 128]."""
    E, rows, K = codes.shape
    t = codes.reshape(E * rows // 128, 128, K // 128, 128).transpose(0, 2, 1, 3)
    return np.ascontiguousarray(t.reshape(-1, 128, 128))
