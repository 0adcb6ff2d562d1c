"""Plain 64-bit forms of the integer and gated products and their gradients,
on the CPU, with bounds on what fp32 may miss.  Not collected by pytest."""
from __future__ import annotations

import numpy as np

from block_ref import U

TINY32 = 2.0 ** -126  # what 2^x and 1/x may flush to zero


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1, e) / (1 + e)


def argument(g, act):
    """z of act(g) = g sigmoid(z), and its derivative."""
    if act == "swiglu":
        return g, np.ones_like(g)
    c = np.sqrt(2 / np.pi)
    return 2 * c * (g + 0.044715 * g ** 3), 2 * c * (1 + 3 * 0.044715 * g ** 2)


def gate(g, u, act):
    return g * sigmoid(argument(g, act)[0]) * u


def gate_error(g, u, act, dg=0.0, du=0.0):
    """What fp32 may miss of act(g) u where g and u are off by dg and du.

    The power 2^(-z log2 e): its exponent is off by two roundings of |z| log2 e
    (of the product, of log2 e), for gelu z itself by five more (its two
    constants, g^2, the sum, the product); the power by 2 U (one step), the sum
    by U, the reciprocal by 2 U, two products by 2 U: (8 + 7 |z|) U relative.
    A sigmoid below 2^-126 may be zero.  |act'| is at most 1.13 everywhere."""
    z = np.minimum(np.abs(argument(g, act)[0]), 120.0)  # past it the sigmoid is 0 or 1
    h = np.abs(gate(g, u, act))
    return (8 + 7 * z) * U * h + TINY32 * np.abs(g * u) + 1.13 * dg * np.abs(u) \
        + (np.abs(g) + dg) * du


def gate_error_fp32_out(g, u, act):
    """What an fp32 H may miss of act(g) u, g and u known: the exponent is carried
    past fp32, so |z| does not enter.  The power is off by 2 U (one step) and U
    (its low part's product and sum), 1 + e and the reciprocal by U each, three
    products by U each: 8 U relative.  A power below 2^-126 may be zero, and a
    result below it a step of 2^-149 off."""
    return 8 * U * np.abs(gate(g, u, act)) + TINY32 * np.abs(g * u) + 2.0 ** -149 * (1 + np.abs(u))


def gate_gradients(dh, g, u, act):
    """(dg, du) of h = act(g) u."""
    z, dz = argument(g, act)
    s, n = sigmoid(z), sigmoid(-z)
    return dh * u * (s + g * s * n * dz), dh * g * s


def gate_gradient_error(dh, g, u, act):
    """What fp32 may miss of them.  sigmoid and 1 - sigmoid as in gate_error; the
    derivative's second term has five products more, the sum one rounding."""
    z, dz = argument(g, act)
    zz = np.minimum(np.abs(z), 120.0)
    s, n = sigmoid(z), sigmoid(-z)
    rel = (16 + 9 * zz) * U
    dg = np.abs(dh * u) * (s + np.abs(g * s * n * dz)) * rel * 2
    tiny = TINY32 * np.abs(dh * u) * (1 + np.abs(g) * (1 + np.abs(dz)))
    return dg + tiny, np.abs(dh * g * s) * rel + TINY32 * np.abs(dh * g)


def product(A, B):
    """(A . B^T, bound on an fp32 sum's error): at most K additions, each a
    rounding (2 U) of a partial sum no larger than the sum of magnitudes."""
    A, B = A.astype(np.float64), B.astype(np.float64)
    return A @ B.T, 2 * U * (A.shape[1] + 16) * (np.abs(A) @ np.abs(B).T)


def integer_product(A, SA, B, SB):
    """C in fp32, bit for bit: the sums are exact, then converted and scaled by
    one rounding each."""
    sums = A.astype(np.int64) @ B.astype(np.int64).T
    with np.errstate(all="ignore"):
        return sums.astype(np.float32) * SA.astype(np.float32)[:, None] * SB.astype(np.float32)[None]


def quantize(x):
    """(codes, scales) of finite rows, bit for bit."""
    x = x.astype(np.float32)
    amax = np.maximum(np.abs(x).max(1) if x.shape[1] else np.zeros(len(x), np.float32),
                      np.float32(2.0 ** -100))
    q = np.rint(x * (np.float32(127) * (np.float32(1) / amax))[:, None])
    return q.astype(np.int8), amax / np.float32(127)


KEPT_HALF_STEP = 2.0 ** -16  # of what a gated product keeps of g and u: fp32 less eight bits


def kept_row(F):
    return 6 * (-(-F // 16) * 16)


def unkept(kept, F):
    """(g, u) of kept rows: planes of upper halves and third bytes."""
    k = np.ascontiguousarray(kept)
    M, fp = len(k), kept_row(F) // 6
    high = k[:, :4 * fp].copy().view(np.uint16).reshape(M, 2, fp)[:, :, :F].astype(np.uint32)
    third = k[:, 4 * fp:6 * fp].reshape(M, 2, fp)[:, :, :F].astype(np.uint32)
    v = (high << 16 | third << 8).astype(np.uint32).view(np.float32).astype(np.float64)
    return v[:, 0], v[:, 1]


def keep(g, u):
    """Kept rows of values that fit (24 bits)."""
    M, F = g.shape
    fp = kept_row(F) // 6
    bits = np.stack([g, u], 1).astype(np.float32).view(np.uint32)
    assert not (bits & 0xFF).any()
    out = np.zeros((M, 6 * fp), np.uint8)
    high = np.zeros((M, 2, fp), np.uint16)
    high[:, :, :F] = bits >> 16
    out[:, :4 * fp] = high.reshape(M, -1).view(np.uint8)
    third = np.zeros((M, 2, fp), np.uint8)
    third[:, :, :F] = bits >> 8 & 0xFF
    out[:, 4 * fp:] = third.reshape(M, -1)
    return out
