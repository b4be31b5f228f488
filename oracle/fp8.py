"""8-bit (e4m3) rows with one scale for each 128 values, in 64 bits: the
quantiser, the matrix product and the expert MLP of the FP8 format, straight
from their definitions (numpy, no code of the CUDA path)."""
from __future__ import annotations

import numpy as np

GROUP = 128
CODE_MAX = 448.0
AMAX_MIN = 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of each code byte: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; 0x7F and 0xFF are NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def e4m3_step(v) -> np.ndarray:
    """Distance between neighbouring e4m3 values around each |v| (at most 448)."""
    a = np.maximum(np.minimum(np.abs(v), CODE_MAX), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def e4m3_round(v) -> np.ndarray:
    """The nearest e4m3 value, ties to even, at most 448; NaN stays NaN."""
    s = e4m3_step(v)
    return np.clip(np.round(np.asarray(v, np.float64) / s) * s, -CODE_MAX, CODE_MAX)


def group_amax(x) -> np.ndarray:
    """[T, K] -> [T, ceil(K/128)]: the largest |x| that is not NaN, at least 2^-100."""
    T, K = x.shape
    nb = -(-K // GROUP)
    a = np.zeros((T, nb * GROUP))
    a[:, :K] = np.where(np.isnan(x), 0.0, np.abs(x))
    return np.maximum(a.reshape(T, nb, GROUP).max(-1), AMAX_MIN)


def spread(s, K) -> np.ndarray:
    """[T, nb] -> [T, K]: each group's value at each of its places."""
    return np.repeat(s, GROUP, axis=1)[:, :K]


def ratios(x) -> np.ndarray:
    """What is rounded to the codes: 448 x / amax of the value's group."""
    with np.errstate(invalid="ignore"):
        return 448.0 * x / spread(group_amax(x), x.shape[1])


def quantize(x):
    """[T, K] float64 -> (code values [T, K], scales [T, ceil(K/128)])."""
    return e4m3_round(ratios(x)), group_amax(x) / CODE_MAX


def dequantize(q, s) -> np.ndarray:
    return q * spread(s, q.shape[1])


def weight(codes, scales) -> np.ndarray:
    """codes [N, K] u8, scales [ceil(N/128), ceil(K/128)] -> float64 [N, K]."""
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), GROUP, 0)[:N], GROUP, 1)[:, :K]
    return e4m3_values()[codes] * s


def row_offsets(H: int, I: int) -> dict:
    """Byte offsets of an expert row: w13 at 0, then w2, s13, s2, end."""
    hb, ib = -(-H // GROUP), -(-I // GROUP)
    up = lambda n: -(-n // 16) * 16  # noqa: E731
    w2 = 2 * I * H
    s13 = w2 + H * I
    s2 = s13 + up(8 * ib * hb)
    return {"w13": 0, "w2": w2, "s13": s13, "s2": s2, "end": s2 + up(4 * ib * hb)}


def expert_weights(row: np.ndarray, H: int, I: int):
    """(gate [I, H], up [I, H], w2 [H, I]) of one expert row, float64."""
    o = row_offsets(H, I)
    hb, ib = -(-H // GROUP), -(-I // GROUP)
    w13 = row[:o["w2"]].reshape(2, I, H)
    s13 = row[o["s13"]:o["s13"] + 8 * ib * hb].view(np.float32).reshape(2, ib, hb)
    w2 = row[o["w2"]:o["s13"]].reshape(H, I)
    s2 = row[o["s2"]:o["s2"] + 4 * ib * hb].view(np.float32).reshape(hb, ib)
    return weight(w13[0], s13[0]), weight(w13[1], s13[1]), weight(w2, s2)


def hidden(xd, gate, up) -> np.ndarray:
    """silu(x gate^T) * (x up^T) of dequantised rows."""
    g = xd @ gate.T
    return g / (1.0 + np.exp(-g)) * (xd @ up.T)


def expert_mlp(xd, row, H, I) -> np.ndarray:
    """Dequantised rows through one expert, h quantised between the products."""
    gate, up, w2 = expert_weights(row, H, I)
    return dequantize(*quantize(hidden(xd, gate, up))) @ w2.T
