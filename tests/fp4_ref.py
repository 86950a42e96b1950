"""A plain reference of the microscaled 4-bit formats in numpy, 64 bits where
the definition does not say 32: quantisation, layouts, values, product."""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BLOCK = {MX: 32, NV: 16}


def pad_up(n, m):
    return (n + m - 1) // m * m


# every finite e4m3 value by its byte (0..126)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest_even(v, grid):
    """Index of the grid value (ascending) nearest to v >= 0; a tie takes the even index; saturates."""
    v = np.minimum(v, grid[-1])
    hi = np.clip(np.searchsorted(grid, v, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def quantise(x, fmt, g=None):
    """x float [rows, K] -> (codes uint8 [rows, K_pad], one code a byte; scale bytes uint8 [rows, K_pad / B])."""
    rows, K = x.shape
    B = BLOCK[fmt]
    Kp = pad_up(K, 128)
    with np.errstate(all="ignore"):
        z = np.zeros((rows, Kp), dtype=np.float32)
        z[:, :K] = x.astype(np.float32)
        if g is not None:
            z *= np.float32(1) / np.float32(g)
        zb = z.reshape(rows, Kp // B, B)
        bad = ~np.isfinite(zb).all(axis=2)
        top = np.abs(np.where(np.isfinite(zb), zb, 0)).max(axis=2).astype(np.float32)
        if fmt == MX:
            e = np.where(top > 0, np.frexp(top.astype(np.float64))[1] - 1 - 2, -127).clip(-127, 127)
            sb = (e + 127).astype(np.uint8)
            s = np.ldexp(1.0, e)
            sb[bad] = 255
        else:
            i = nearest_even(top.astype(np.float64) / 6.0, E4M3)
            sb = i.astype(np.uint8)
            s = E4M3[i]
            sb[bad] = 127
        s = np.where(bad, 0.0, s)
        q = np.abs(np.where(np.isfinite(zb), zb, 0).astype(np.float64)) / np.where(s > 0, s, 1.0)[..., None]
        c = nearest_even(q, GRID).astype(np.uint8)
        c[s == 0] = 0
        c |= (np.signbit(zb) & ~bad[..., None]).astype(np.uint8) << 3
    return c.reshape(rows, Kp), sb


def pack(codes, sb, fmt):
    """(code rows uint8 [rows, K_pad / 2], scale tiles uint8 [bytes]) in the library's layout."""
    rows, Kp = codes.shape
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    nb = sb.shape[1]
    t = np.zeros((pad_up(rows, 128), nb), dtype=np.uint8)
    t[:rows] = sb
    out = np.zeros(t.size, dtype=np.uint8)
    r, c = np.meshgrid(np.arange(t.shape[0]), np.arange(nb), indexing="ij")
    out[((r // 128) * (nb // 4) + c // 4) * 512 + 16 * (r % 32) + 4 * ((r % 128) // 32) + c % 4] = t
    return packed, out


def scale_values(sb, fmt):
    if fmt == MX:
        return np.where(sb == 255, np.nan, np.ldexp(1.0, sb.astype(np.int64) - 127))
    return np.where((sb & 127) == 127, np.nan, E4M3[np.minimum(sb & 127, 126)] * np.where(sb & 128, -1.0, 1.0))


def values(codes, sb, fmt):
    """element * scale in 64 bits, [rows, K_pad]."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(scale_values(sb, fmt), BLOCK[fmt], axis=1)


def random_matrix(rows, K, fmt, rng, spread=3):
    """Random codes and scales around 1: (codes [rows, K_pad] with code 0 past K, scale bytes)."""
    Kp = pad_up(K, 128)
    codes = rng.integers(0, 16, (rows, Kp), dtype=np.uint8)
    codes[:, K:] = 0
    nb = Kp // BLOCK[fmt]
    if fmt == MX:
        sb = rng.integers(127 - spread, 127 + spread, (rows, nb)).astype(np.uint8)
    else:
        sb = rng.integers(56 - 8 * spread, 56 + 8 * spread, (rows, nb)).astype(np.uint8)
    return codes, sb


def product(av, wv, scale=1.0):
    """(A W^T scale, sum |a||w| scale) in 64 bits."""
    return av @ wv.T * scale, np.abs(av) @ np.abs(wv).T * abs(scale)


def product_tolerance(y, mag, K, eps):
    """Half a step of the output's type, and what the fp32 sums may lose: K / 16 additions and the few of the
    blocks that are put together, each off by at most 2^-22 (a truncated fp32 step) of the sum of magnitudes;
    then two roundings of the product with the tensor scales."""
    return eps / 2 * np.abs(y) * (1 + 2.0 ** -20) + mag * ((K / 16 + 16) * 2.0 ** -22 + 2.0 ** -22)
