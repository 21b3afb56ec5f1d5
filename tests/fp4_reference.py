"""The 4-bit formats' definition in numpy, with the fp32 roundings that it
names, for the tests: quantisation, the packed layouts, and the product in 64
bits.  Shares no code with the library."""
import numpy as np

NV, MX = 0, 1
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([MAGNITUDES, -MAGNITUDES])


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = -m if c & 128 else m
    v[127] = v[255] = np.nan
    return v


E4M3 = _e4m3_table()


def _nearest(q, grid):
    """Index of the grid value nearest to q >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, q, side="left"), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = q - grid[lo], grid[hi] - q
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return np.where((hi == lo) | up | (q >= grid[-1]), hi, lo)


def quantise(v, fmt):
    """fp32 rows [R, K] -> (codes uint8 [R, K] without the sign of zeros, scale
    bytes uint8 [R, K / 16 or 32], row scales fp32 [R])."""
    v = np.asarray(v, np.float32)
    R, K = v.shape
    blk = 16 if fmt == NV else 32
    b = v.reshape(R, K // blk, blk)
    am = np.abs(b).max(axis=2)
    if fmt == NV:
        r = (np.abs(v).max(axis=1) / np.float32(2688)).astype(np.float32)
        r = np.where(r < np.float32(2.0 ** -126), np.float32(1), r)
        s = ((am / np.float32(6)).astype(np.float32) / r[:, None]).astype(np.float32)
        byte = _nearest(s.astype(np.float64), E4M3[:127])
        d = (E4M3[byte].astype(np.float32) * r[:, None]).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(d[:, :, None] > 0, (b / d[:, :, None]).astype(np.float32), np.float32(0))
    else:
        e = np.where(am > 0, np.frexp(am)[1] - 3, 0).clip(-127, 127)
        byte = e + 127
        q = b.astype(np.float64) * 2.0 ** (-e.astype(np.float64))[:, :, None]
        r = np.ones(R, np.float32)
    code = _nearest(np.abs(q).astype(np.float64), MAGNITUDES)
    code = np.where((q < 0) & (code > 0), code + 8, code)
    return code.reshape(R, K).astype(np.uint8), byte.astype(np.uint8), r


def values(codes, byte, r, fmt, dtype=np.float64):
    """The values that codes stand for; np.float32 rounds as fp4_dequant_weights does."""
    s = E4M3[byte] if fmt == NV else 2.0 ** (byte.astype(np.float64) - 127)
    d = s.astype(dtype) * r.astype(dtype)[:, None]
    v = E2M1[codes].astype(dtype).reshape(*d.shape, -1) * d[:, :, None]
    return v.reshape(codes.shape).astype(dtype)


def pack_codes(codes, tiled):
    """Codes [R, K] -> the packed bytes: [tiles, 128, 128] (weights) or [R, kt * 128]."""
    R, K = codes.shape
    kt = -(-K // 256)
    rows = -(-R // 128) * 128 if tiled else R
    p = np.zeros((rows, kt * 256), np.uint8)
    p[:R, :K] = codes
    b = p[:, 0::2] | (p[:, 1::2] << 4)
    return b.reshape(rows // 128, 128, kt, 128).transpose(0, 2, 1, 3).reshape(-1, 128, 128) if tiled else b


def pack_atoms(byte, K, fmt):
    """Scale bytes [R, blocks] -> [atoms, 512], rows past R zero."""
    R = byte.shape[0]
    kt = -(-K // 256)
    nb = kt * (16 if fmt == NV else 8)
    p = np.zeros((-(-R // 128) * 128, nb), np.uint8)
    p[:R, :byte.shape[1]] = byte
    out = np.zeros((p.shape[0] // 128, nb // 4, 512), np.uint8)
    for r in range(128):
        for j in range(4):
            out[:, :, 16 * (r % 32) + 4 * (r // 32) + j] = p[r::128, j::4]
    return out.reshape(-1, 512)


def without_zero_signs(packed):
    """Packed bytes with every code 8 (a negative zero) as 0."""
    lo, hi = packed & 15, packed >> 4
    return np.where(lo == 8, 0, lo) | (np.where(hi == 8, 0, hi) << 4)
