"""Plain float64 restatement of the 4-bit latent cache (test infrastructure only): what its bytes stand for, and which
bytes a row of values becomes.  Layout and rounding as the public header states them; attention over the cache is
mla.py's over the values.
"""
from __future__ import annotations

import numpy as np

from .mla import D_LATENT, D_QK, E4M3_VALUES, e4m3_round

ROW_BYTES, GROUP, SCALE_AT, ROPE_AT = 352, 16, 256, 288


def e2m1_value(code: int) -> float:
    """The number a 4-bit E2M1 code stands for: a sign, two exponent bits with bias 1, one mantissa bit."""
    sign, e, m = code >> 3 & 1, code >> 1 & 3, code & 1
    v = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -v if sign else v


E2M1_VALUES = np.array([e2m1_value(i) for i in range(16)])
E2M1_MIDDLES = (E2M1_VALUES[:7] + E2M1_VALUES[1:8]) / 2      # between codes i and i + 1


def e2m1_round(v) -> np.ndarray:
    """E2M1 codes (uint8) of float values: the nearest number, halfway to the even code, beyond +-6 the largest one.  A
    negative value that rounds to zero keeps its sign; NaN gives 0."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    code = np.zeros(v.shape, dtype=np.uint8)
    for i, mid in enumerate(E2M1_MIDDLES):
        code += (a > mid) if i % 2 == 0 else (a >= mid)      # halfway: down to the even i, or up to the even i + 1
    return code | np.where(np.signbit(v) & ~np.isnan(v), 8, 0).astype(np.uint8)


def pack_fp4(rows, kv_scale) -> np.ndarray:
    """[..., 576] values as [..., 352] bytes."""
    x = np.asarray(rows, dtype=np.float64)
    assert x.shape[-1] == D_QK
    unit = float(np.float32(kv_scale))
    g = x[..., :D_LATENT].reshape(*x.shape[:-1], D_LATENT // GROUP, GROUP)
    scale = e4m3_round(np.abs(g).max(axis=-1) / (6.0 * unit))     # (NaN in a group: the NaN code)
    step = E4M3_VALUES[scale] * unit
    ok = (step > 0)[..., None]
    with np.errstate(invalid="ignore"):
        code = np.where(ok, e2m1_round(g / np.where(ok, step[..., None], 1.0)), 0).reshape(*x.shape[:-1], D_LATENT)
    code = code.astype(np.uint8)
    rope = e4m3_round(x[..., D_LATENT:] / unit)
    return np.concatenate((code[..., 0::2] | code[..., 1::2] << 4, scale, rope), axis=-1).astype(np.uint8)


def unpack_fp4(data, kv_scale) -> np.ndarray:
    """[..., 352] bytes as the [..., 576] values they stand for."""
    data = np.asarray(data)
    assert data.shape[-1] == ROW_BYTES
    low, high = E2M1_VALUES[data[..., :SCALE_AT] & 15], E2M1_VALUES[data[..., :SCALE_AT] >> 4]
    code = np.stack((low, high), axis=-1).reshape(*data.shape[:-1], D_LATENT)
    scale = np.repeat(E4M3_VALUES[data[..., SCALE_AT:ROPE_AT]], GROUP, axis=-1)
    return np.concatenate((code * scale, E4M3_VALUES[data[..., ROPE_AT:]]), axis=-1) * float(np.float32(kv_scale))


def normed_latent(c, weight, eps) -> np.ndarray:
    """c * rsqrt(mean(c^2) + eps) * weight, row by row."""
    c = np.asarray(c, dtype=np.float64)
    return c / np.sqrt((c * c).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
