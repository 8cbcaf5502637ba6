"""The 4-bit microscaled formats in plain numpy, 64 bits, written from their
definitions: E2M1 codes, E4M3 / E8M0 block scales, the stored scale layout,
quantisation, and operands made of random codes and scales.

Tolerances of the GPU tests.  Product: a code product is a multiple of 1/4 up
to 36 and every scale product has at most 8 significant bits, so each term is
exact in fp32; the sum follows the rule of every parity test of this library
(1e-5 * S + 1e-6, S the sum of magnitudes, plus one ulp of a 16-bit D).
Quantisation of a given tensor is exact: codes and scale bytes are compared
for equality.
"""
import numpy as np

MXFP4, NVFP4 = 1, 2
BLOCK = {MXFP4: 32, NVFP4: 16}
MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAG, -MAG])


def ceil(a, b):
    return -(-a // b)


def e4m3_values():
    """Value of every byte 0..127 (sign clear); byte 127 is NaN."""
    b = np.arange(128)
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return v


def scale_values(byte, fmt):
    byte = np.asarray(byte).astype(np.int64)
    if fmt == NVFP4:
        return e4m3_values()[byte & 127]
    return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))


def nearest(table, x):
    """Index of the nearest entry of an ascending table; ties to the even
    index; beyond the ends, the end."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(pick_hi, hi, lo)


def quantize(x, fmt, g=1.0):
    """fp64 [rows, k] -> codes [rows, k], scale bytes [rows, blocks]."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    b = BLOCK[fmt]
    nb = ceil(k, b)
    v = np.zeros((rows, nb * b))
    v[:, :k] = x
    v = v.reshape(rows, nb, b)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(-1)
        bad = ~np.isfinite(v).all(-1)
        amax = np.where(bad, 0.0, amax)
        if fmt == NVFP4:
            byte = nearest(e4m3_values()[:127], amax / (6.0 * g))
            s = e4m3_values()[byte] * g
            byte = np.where(bad, 127, byte)
        else:
            e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1
            byte = np.where(amax > 0, np.clip(e - 2 + 127, 0, 254), 0)
            s = 2.0 ** (byte - 127.0)
            byte = np.where(bad, 255, byte)
        live = ((s > 0) & ~bad)[..., None]
        w = np.where(live, v / np.where(s > 0, s, 1.0)[..., None], 0.0)
    code = nearest(MAG, np.abs(w)) + 8 * np.signbit(w)
    return code.reshape(rows, -1)[:, :k].astype(np.uint8), byte.astype(np.uint8)


def pack(code, ld=None):
    """[..., rows, k] codes -> [..., rows, ld / 2] bytes."""
    k = code.shape[-1]
    ld = ceil(k, 32) * 32 if ld is None else ld
    full = np.zeros(code.shape[:-1] + (ld,), dtype=np.uint8)
    full[..., :k] = code
    return full[..., 0::2] | (full[..., 1::2] << 4)


def unpack(packed, k):
    out = np.stack([packed & 15, packed >> 4], -1)
    return out.reshape(packed.shape[:-1] + (-1,))[..., :k]


def scale_at(r, b, atoms):
    return ((r // 128) * atoms + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def tile(byte, row=None, tiles=None, fill=0):
    """Scale bytes [rows, blocks] -> the stored bytes; row[i]: scale row of row
    i.  Padding blocks of a stored row are zero, rows not held are `fill`."""
    rows, nb = byte.shape
    row = np.arange(rows) if row is None else np.asarray(row)
    tiles = ceil(rows, 128) if tiles is None else tiles
    atoms = ceil(nb, 4)
    flat = np.full(tiles * atoms * 512, fill, dtype=np.uint8)
    full = np.zeros((rows, atoms * 4), dtype=np.uint8)
    full[:, :nb] = byte
    flat[scale_at(row[:, None], np.arange(atoms * 4)[None], atoms)] = full
    return flat


def expert_rows(offsets):
    """Scale row of every token row: each expert starts on an atom row."""
    start, out = 0, []
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        out.append(start * 128 + np.arange(hi - lo))
        start += ceil(hi - lo, 128)
    return np.concatenate(out).astype(np.int64)


def dequantize(code, byte, fmt, g=1.0):
    s = np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=-1)[..., :code.shape[-1]]
    return VALUES[code] * s * g


def random_operand(rng, rows, k, fmt):
    """Every code; scales over a few binades."""
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    nb = ceil(k, BLOCK[fmt])
    byte = rng.integers(40, 64, (rows, nb)) if fmt == NVFP4 else rng.integers(123, 131, (rows, nb))
    return code, byte.astype(np.uint8)
