"""Microscaled formats in 64 bits, for the tests: written from the definition
(element grids enumerated, nearest one taken), apart from the library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]
GRID = {"mxfp4": E2M1, "mxfp8": E4M3}


def nearest(v, grid):
    """Index of the grid value nearest to each |v|, a tie to the even index."""
    v = np.abs(v)
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantize(x, fmt):
    """(signed element values, scale bytes, codes) of x [rows, K]."""
    rows, K = x.shape
    grid = GRID[fmt]
    b = x.reshape(rows, K // 32, 32)
    with np.errstate(invalid="ignore"):
        big = np.abs(b).max(-1)
    bad = ~np.isfinite(big)
    safe = np.where(bad, 0, big)
    byte = np.zeros(big.shape, dtype=int)
    for e in range(254):            # the least exponent with which nothing saturates
        byte += safe > grid[-1] * 2.0 ** (e - 127)
    byte[bad] = 255
    scaled = np.where(bad[..., None], 0, b) * 2.0 ** (127.0 - np.where(bad, 127, byte))[..., None]
    code = nearest(scaled, grid)
    value = np.copysign(grid[code], scaled)
    sign = np.signbit(scaled) & ~bad[..., None]
    return value.reshape(rows, K), byte, (code + sign * len_sign(fmt)).reshape(rows, K)


def len_sign(fmt):
    return 8 if fmt == "mxfp4" else 128


def values(element, byte):
    """element * 2^(byte - 127), NaN for byte 255."""
    s = np.where(byte == 255, np.nan, 2.0 ** (np.where(byte == 255, 0, byte) - 127.0))
    return (element.reshape(*byte.shape, 32) * s[..., None]).reshape(element.shape)


def tiled(byte):
    """Row-major scale bytes in the library's tile order, zeros past the end."""
    rows, blocks = byte.shape
    R, B = -(-rows // 128), -(-blocks // 4)
    out = np.zeros((R, B, 32, 4, 4), dtype=np.uint8)
    for r in range(rows):
        for k in range(blocks):
            out[r // 128, k // 4, r % 32, r % 128 // 32, k % 4] = byte[r, k]
    return out
