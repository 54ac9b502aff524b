"""The microscaled 4-bit formats from their definition, in float64 numpy: used by the tests of
quantize / dequantize and of the 4-bit projections.  Rounding is by comparison with the midpoints of
a table of the format's values (a tie goes to the even code), so no arithmetic rounds."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])  # codes 0 .. 126
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def nearest(v, table):
    """Index of the table value nearest to v >= 0; the last one above the table."""
    mid = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mid, v, side="left")   # midpoints < v
    hi = np.searchsorted(mid, v, side="right")  # midpoints <= v
    return np.where(lo % 2 == 0, lo, hi)        # (they differ on a tie only: the even one of lo, lo + 1)


def scale_tiles(fmt, K):
    return -(-K // (4 * BLOCK[fmt]))


def quantize(x, fmt):
    """codes [rows, K] (0..15), scale codes [rows, K / B], row scales [rows] of x (float64 [rows, K])."""
    rows, K = x.shape
    B = BLOCK[fmt]
    blocks = np.abs(x).reshape(rows, K // B, B)
    bad = ~np.isfinite(x).all(1)
    blocks = np.where(bad[:, None, None], 0.0, blocks)
    top = blocks.max(2)
    if fmt == "nvfp4":
        amax = top.max(1)
        row = np.array([2.0 ** max(-100, next((j for j in range(-101, 128) if a <= 2688.0 * 2.0 ** j))) for a in amax])
        # top / (6 g) against E4M3: both sides times 6 g, exact
        sc = nearest(top / row[:, None], 6 * E4M3)
        s = E4M3[sc] * row[:, None]
    else:
        row = np.ones(rows)
        e = np.where(top > 0, np.frexp(top)[1] - 3, -127)
        sc = np.maximum(e, -127) + 127
        s = 2.0 ** (sc - 127.0)
    q = np.where(s[..., None] > 0, blocks / np.where(s > 0, s, 1.0)[..., None], 0.0)
    codes = nearest(q, E2M1).reshape(rows, K)
    codes = np.where(np.signbit(x) & ~bad[:, None], codes + 8, codes)
    sc = np.where(bad[:, None], 0, sc)
    return codes, sc, np.where(bad, np.nan, row)


def values(codes, sc, row, fmt):
    B = BLOCK[fmt]
    s = E4M3[sc] if fmt == "nvfp4" else 2.0 ** (sc - 127.0)
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(s, B, axis=1) * row[:, None]


def unpack(q):
    """(codes, scale codes, row scales) of a QuantTensor, from the documented layout."""
    rows, K = q.shape
    packed = q.codes.cpu().numpy()
    codes = np.empty((rows, K), np.int64)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    nb = K // BLOCK[q.format]
    flat = q.scales.cpu().numpy().reshape(-1)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    at = ((r // 128) * scale_tiles(q.format, K) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return codes, flat[at].astype(np.int64), q.row_scale.cpu().numpy().astype(np.float64)
