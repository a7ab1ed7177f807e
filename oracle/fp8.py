"""8-bit KV cache blocks: e4m3 codes with a power-of-two scale per 32 tokens.

Test infrastructure only (see ``oracle/__init__.py``).  The pages name a 4-bit
KV cache only; this is the reading of an 8-bit one that ``duo.h`` states: per
(KV head, 32 consecutive tokens), K and V apart,

    sc = 2^e, e the smallest integer >= -120 with max|x| <= 448 * 2^e  (finite x)
    code = e4m3 nearest to x / sc, ties to even, saturating at +-448, NaN kept
           (at sc = 2^120 at +-240: a code of 256 would stand for 2^128, past
           float32's range)
    x_hat = sc * code                                (exact in fp64)

and tokens past the last full block are held as they are.  e4m3 has no
infinity: 4 significant bits from 2^-6 up to 448, steps of 2^-9 below.
"""

import numpy as np

__all__ = ["BLOCK", "block_scale", "nearest_e4m3", "encode_e4m3", "held"]

BLOCK = 32


def block_scale(x):
    """x [..., BLOCK, d] float64 -> scale [...]."""
    a = np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=(-1, -2))
    m, ex = np.frexp(a)  # a = m * 2^ex, m in [0.5, 1)
    e = np.where(m > 448.0 / 512.0, ex - 8, ex - 9)
    e = np.where(a > 0, e, -120)
    return np.exp2(np.maximum(e, -120).astype(np.float64))


def nearest_e4m3(z):
    """The e4m3 value nearest to each z (ties to even), saturating."""
    z = np.clip(np.asarray(z, np.float64), -448.0, 448.0)
    _, ex = np.frexp(np.maximum(np.abs(z), 2.0 ** -6))
    step = np.exp2((ex - 4).astype(np.float64))
    return np.rint(z / step) * step


def encode_e4m3(v):
    """The byte of each e4m3 value v (sign, 4 exponent bits of bias 7, 3 mantissa bits)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    _, ex = np.frexp(np.maximum(a, 2.0 ** -6))
    e = ex - 1
    normal = a >= 2.0 ** -6
    mant = np.where(normal, (a / np.exp2(e.astype(np.float64)) - 1.0) * 8.0, a * 2.0 ** 9)
    code = np.where(normal, (e + 7) * 8, 0) + mant
    code = np.where(np.isnan(v), 0x7F, code)
    return (code.astype(np.uint8) | (np.signbit(v) & ~np.isnan(v)).astype(np.uint8) << 7).astype(np.uint8)


def held(x):
    """What the cache holds of one row's tokens x [n, heads, d]: float64, full
    blocks through the codes, later tokens as they are.  Also the code values
    [blocks * BLOCK, heads, d] and the scales [blocks, heads]."""
    x = np.asarray(x, np.float64)
    n, heads, d = x.shape
    full = n // BLOCK * BLOCK
    out = x.copy()
    if full == 0:
        return out, np.zeros((0, heads, d)), np.zeros((0, heads))
    y = x[:full].reshape(-1, BLOCK, heads, d).transpose(0, 2, 1, 3)  # [blocks, heads, BLOCK, d]
    sc = block_scale(y)
    codes = nearest_e4m3(y / sc[..., None, None])
    top = (sc == 2.0 ** 120)[..., None, None]
    codes = np.where(top, np.clip(codes, -240.0, 240.0), codes)
    out[:full] = (codes * sc[..., None, None]).transpose(0, 2, 1, 3).reshape(full, heads, d)
    return out, codes.transpose(0, 2, 1, 3).reshape(full, heads, d), sc
