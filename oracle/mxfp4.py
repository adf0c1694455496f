"""MXFP4 operands in float64 (oracle; test infrastructure), from the definition.

OCP MX v1.0 MXFP4: groups of 32 elements share the scale 2^e, e = floor(log2 amax) - 2 clamped to [-127, 127] (2 is the
exponent of E2M1's largest binade, 4 to 6); an element is the E2M1 number nearest to v / 2^e, ties to the even code,
saturated to 6, the sign kept. Readings, as for MXFP8: a group with amax 0 has scale byte 0; one that holds a NaN or an
infinity has byte 255 and reads back as NaN.

Operand of [rows, K]: codes [P, rows, 64], scales [P, rows, 4], P = ceil(K / 128), the contraction padded with zeros; E2M1
codes two to a byte, the lower k in the lower four bits; E4M3 codes [2 P, rows, 64].
"""
import numpy as np

from .formats import e4m3_to_f64, e8m0_to_f64
from .mx import quantize_blocks, scale_byte

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_to_f64(c):
    c = np.asarray(c)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def to_e2m1(v):
    """Codes of the E2M1 numbers nearest to v (finite), ties to the even code, saturated."""
    v = np.asarray(v, dtype=np.float64)
    m = np.abs(v)
    hi = np.clip(np.searchsorted(E2M1, m), 1, 7)
    lo = hi - 1
    mid = (E2M1[lo] + E2M1[hi]) / 2
    up = (m > mid) | ((m == mid) & (hi % 2 == 0))
    return (np.where(up, hi, lo) + np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def quantize_groups(v):
    """E2M1 codes and scale bytes of groups v [..., 32]."""
    v = np.asarray(v, dtype=np.float64)
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    byte = np.where(bad, 255, np.where(amax == 0, 0, scale_byte(amax, emax=2))).astype(np.uint8)
    safe = np.where(bad[..., None], 0.0, v)
    scale = np.where(bad, 1.0, e8m0_to_f64(np.where(bad, 127, byte).astype(np.uint8)))
    return to_e2m1(safe / scale[..., None]), byte


def operand(v, e4m3=False):
    """(q, s) of v [rows, K]."""
    v = np.asarray(v, dtype=np.float64)
    rows, K = v.shape
    P = -(-K // 128)
    p = np.zeros((rows, P * 128))
    p[:, :K] = v
    p = p.reshape(rows, P * 4, 32)
    q, s = (quantize_blocks if e4m3 else quantize_groups)(p)
    s = s.reshape(rows, P, 4).transpose(1, 0, 2)
    q = q.reshape(rows, P * 128)
    if not e4m3:
        q = q[:, 0::2] | q[:, 1::2] << 4
    return np.ascontiguousarray(q.reshape(rows, -1, 64).transpose(1, 0, 2)), np.ascontiguousarray(s)


def values(q, s):
    """The float64 matrix [rows, 128 P] of an operand."""
    P, rows, _ = s.shape
    c = q.transpose(1, 0, 2).reshape(rows, -1)
    if q.shape[0] == P:
        c = np.stack([c & 15, c >> 4], 2).reshape(rows, -1)
        v = e2m1_to_f64(c)
    else:
        v = e4m3_to_f64(c)
    return v * np.repeat(e8m0_to_f64(s.transpose(1, 0, 2).reshape(rows, -1)), 32, axis=1)
