"""fp64 oracle of MXFP4 (OCP Microscaling Formats v1.0): plain numpy, by comparison of distances.

A block is 32 consecutive values of a row; a value is level(code) * 2^(s - 127) with the E2M1
levels below, negative where bit 3 of the code is set, NaN throughout where s = 255.
"""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pitch(k: int) -> int:
    return (k + 511) // 512 * 16


def quantize(x: np.ndarray):
    """x [n, k] (any float type, taken as it is) -> (codes uint8 [n, k], scale uint8 [n, pitch(k)])."""
    v = np.asarray(x, dtype=np.float64)
    n, k = v.shape
    v = v.reshape(n, k // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1)
    floor_log2 = np.frexp(amax)[1] - 1                       # amax = m 2^e, m in [1/2, 1)
    e = np.where(amax > 0, np.maximum(floor_log2 - 2, -127), -127)
    a = np.ldexp(np.abs(v), -e[..., None])
    dist = np.abs(a[..., None] - LEVELS)
    least = dist.min(-1, keepdims=True)
    # the nearest level; of two equally near ones the even code
    rank = np.where(dist == least, np.arange(8) % 2, 2)
    code = rank.argmin(-1).astype(np.uint8)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    scale = np.zeros((n, pitch(k)), np.uint8)
    scale[:, :k // 32] = np.where(bad, 255, e + 127)
    return code.reshape(n, k), scale


def values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The float64 [n, k] values of codes and scale bytes."""
    n, k = codes.shape
    lv = np.where(codes & 8, -LEVELS[codes & 7], LEVELS[codes & 7]).reshape(n, k // 32, 32)
    s = scale[:, :k // 32].astype(np.int64)
    with np.errstate(invalid="ignore"):
        out = np.ldexp(lv, (s - 127)[..., None])
    return np.where((s == 255)[..., None], np.nan, out).reshape(n, k)


def product(xv: np.ndarray, wv: np.ndarray):
    """(x W^T, |x| |W|^T) in float64."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T
