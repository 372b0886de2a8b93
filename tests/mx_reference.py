"""Blocks of 32 values with a power of two, in numpy and 64 bits: what the tests of them compare with."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
TOP = {4: 2, 8: 8}
LARGEST = {4: 6.0, 8: 448.0}


def code_values(bits):
    """The value of every code."""
    if bits == 4:
        return np.concatenate([E2M1, -E2M1])
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e > 0, np.ldexp(1 + m / 8, e - 7), np.ldexp(m / 8, -6))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


def powers(byte):
    byte = np.asarray(byte).astype(np.int64)
    return np.where(byte == 255, np.nan, np.ldexp(1.0, np.minimum(byte, 254) - 127))


def step_at(u, bits):
    """The distance between neighbouring values of the type around u."""
    smallest, mantissa = (0, 1) if bits == 4 else (-6, 3)
    return np.ldexp(1.0, np.maximum(np.frexp(np.abs(u))[1] - 1, smallest) - mantissa)


def nearest(u, bits):
    """To the type's nearest value, ties to even, clipped."""
    s = step_at(u, bits)
    return np.clip(np.rint(u / s) * s, -LARGEST[bits], LARGEST[bits])


def block_bytes(v, bits):
    """The power's byte of each block of v [m, k] (float64)."""
    m, k = v.shape
    top = np.abs(v).reshape(m, k // 32, 32)
    fine = np.isfinite(top).all(axis=-1)
    top = np.where(fine, np.where(np.isfinite(top), top, 0).max(axis=-1), 0.0)
    power = np.where(top > 0, np.frexp(top)[1] - 1 - TOP[bits], -127)
    return np.where(fine, np.maximum(power, -127) + 127, 255).astype(np.uint8)


def blocks(v, bits):
    """Values q [m, k] (without their powers) and bytes [m, k / 32] of v in float64."""
    m, k = v.shape
    byte = block_bytes(v, bits)
    bad = byte == 255
    u = np.where(bad[:, :, None], 0.0, v.reshape(m, k // 32, 32)) / powers(np.where(bad, 127, byte))[:, :, None]
    return nearest(u, bits).reshape(m, k), byte


def unpack(codes, bits):
    """uint8 [m, bytes] to the values of the codes [m, k]."""
    if bits == 8:
        return code_values(8)[codes]
    both = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    return code_values(4)[both]


def expanded(codes, byte, bits):
    """What codes [m, bytes] with bytes [m, k / 32] stand for, in float64."""
    v = unpack(codes, bits)
    return v * np.repeat(powers(byte), 32, axis=1)
