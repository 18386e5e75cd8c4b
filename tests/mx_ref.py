"""Plain double-precision definitions of the microscaled operators (numpy),
written from the formats alone."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                 for e in range(16) for m in range(8)][:127], np.float64)      # 448 is code 126
MXFP4, MXFP8 = 0, 1
GRID, TOP = {MXFP4: E2M1, MXFP8: E4M3}, {MXFP4: 6.0, MXFP8: 448.0}


def nearest(grid, a):
    """Index of the grid value nearest to a >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    dh, dl = grid[hi] - a, a - grid[hi - 1]
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)


def scale_exponent(m, fmt):
    """Smallest e >= -127 with m <= TOP 2^e (m > 0, finite)."""
    f, e = np.frexp(m / TOP[fmt])
    return np.maximum(np.where(f == 0.5, e - 1, e), -127)


def quantize(x, fmt):
    """(code index with its sign in the top bit of the code, scale bytes) of
    double rows that hold fp32 values."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    m = np.abs(b).max(-1)
    bad = ~np.isfinite(m)
    e = np.where(bad | (m == 0), -127, scale_exponent(np.where(bad | (m == 0), 1.0, m), fmt))
    a = np.where(bad[..., None], 0.0, np.abs(b)) / np.exp2(e.astype(np.float64))[..., None]
    code = nearest(GRID[fmt], a)
    top = 8 if fmt == MXFP4 else 128
    code = np.where(bad[..., None], 0, code + np.where(np.signbit(b), top, 0)).astype(np.uint8)
    return code.reshape(rows, cols), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code):
    """e2m1 codes [.., cols] to bytes [.., cols/2], the low nibble the even column."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(code, scales, fmt):
    """Doubles that codes (unpacked) and scale bytes stand for."""
    top = 8 if fmt == MXFP4 else 128
    mag = code % top
    v = GRID[fmt][np.minimum(mag, len(GRID[fmt]) - 1)]
    if fmt == MXFP8:
        v = np.where(mag == 127, np.nan, v)
    v = np.where(code >= top, -v, v)
    v = v.reshape(*scales.shape, 32) * np.exp2(scales.astype(np.float64) - 127.0)[..., None]
    v = np.where((scales == 255)[..., None], 0.0 if fmt == MXFP4 else np.nan, v)
    return v.reshape(code.shape)


def product(xcode, xs, packed, ws):
    """(y, sum |x w|) in double."""
    x, w = values(xcode, xs, MXFP8), values(unpack(packed), ws, MXFP4)
    return x @ w.T, np.abs(x) @ np.abs(w).T
