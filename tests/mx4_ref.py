"""The microscaled 4-bit format and its product, written down plainly in 64 bits
(numpy; no code of the library)."""
import math

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def encode(x):
    """x [rows, K] (float64 holding bf16 values) -> codes [rows, K] (0..15), scale bytes [rows, ceil(K/32)]."""
    rows, K = x.shape
    nblk = -(-K // 32)
    p = np.zeros((rows, nblk * 32))
    p[:, :K] = x
    p = p.reshape(rows, nblk, 32)
    codes = np.zeros(p.shape, np.uint8)
    scales = np.zeros((rows, nblk), np.uint8)
    for r in range(rows):
        for b in range(nblk):
            v = p[r, b]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                continue
            amax = np.abs(v).max()
            e = -127 if amax == 0 else max(math.frexp(amax)[1] - 3, -127)
            scales[r, b] = e + 127
            a = np.abs(v) / 2.0 ** e
            d = np.abs(a[:, None] - GRID)
            near = d.min(1, keepdims=True)
            # of two equally near values, the one with the even code
            tie = (d == near)
            code = np.where(tie.sum(1) == 2, (tie * (np.arange(8) % 2 == 0)).argmax(1), tie.argmax(1))
            codes[r, b] = code + 8 * np.signbit(v)
    return codes.reshape(rows, -1)[:, :K], scales


def pack_codes(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack_codes(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def values(codes, scales):
    """What codes [rows, K] and scale bytes stand for, float64."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)[:, : codes.shape[1]]


def sum_error(a, w, K):
    """A bound on the error of an fp32 sum of the K products of a [M, K] and w [N, K] on the tensor core:
    K / 64 instructions, each adding 64 exact products to the running sum with at most a few roundings
    or truncations (2^-23) relative to the sum of magnitudes."""
    return (K / 64 + 8) * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T)


def gelu(t):
    """0.5 t (1 + tanh u) as t / (1 + e^(-2u)): the sum 1 + tanh u is 0 in 64 bits from u = -19 on."""
    with np.errstate(over="ignore"):
        return t / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
