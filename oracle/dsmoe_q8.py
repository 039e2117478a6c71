"""Float64 definitions of the 8-bit path, in numpy: the 8-bit form of a matrix (e4m3 values
with one power of two per block of 128), the RMSNorm with the residual's addition and its
backward pass, and the grouped products. Independent of the CUDA library; test
infrastructure only."""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def scale_cols(C: int) -> int:
    return 4 * (-(-C // 512))


def e4m3_values() -> np.ndarray:
    """The 256 values of the format: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and
    0xFF are NaN, there are no infinities."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[b] = np.nan if (e == 15 and m == 7) else v
        if b & 128:
            out[b] = -out[b]
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # 0 .. 448, increasing


def encode_e4m3(v) -> np.ndarray:
    """Bytes of the nearest e4m3 values (ties to the even mantissa), |v| <= 448; NaN gives 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _POSITIVE[lo], _POSITIVE[hi] - a
    take_hi = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    code = np.where(take_hi, hi, lo).astype(np.uint8)
    code = np.where(np.signbit(v), code | 128, code)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def decode_e4m3(b) -> np.ndarray:
    return _VALUES[np.asarray(b)]


def decode_scale(b) -> np.ndarray:
    b = np.asarray(b).astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def scale_byte(amax) -> np.ndarray:
    """Byte of the smallest 2^k >= amax / 448 with k >= -126; 255 for an infinite or NaN maximum."""
    amax = np.asarray(amax, dtype=np.float64)
    fine = np.isfinite(amax)
    k = np.full(amax.shape, -126, dtype=np.int64)
    while True:  # one step of two at a time: the definition, not a logarithm
        low = fine & (amax > E4M3_MAX * np.ldexp(1.0, k))
        if not low.any():
            break
        k = np.where(low, k + 1, k)
    return np.where(fine, k + 127, 255).astype(np.uint8)


def _encode_blocks(x, byte):
    """Bytes of x under the (already broadcast) scale bytes."""
    with np.errstate(invalid="ignore"):
        v = np.where(byte == 255, np.nan, x / np.where(byte == 255, 1.0, decode_scale(np.minimum(byte, 254))))
    return encode_e4m3(v)


def quantize_rows(x):
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    nb = -(-C // BLOCK)
    q = np.empty((R, C), np.uint8)
    s = np.full((R, scale_cols(C)), 127, np.uint8)
    for b in range(nb):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b] = scale_byte(np.abs(part).max(axis=1) if R else np.zeros(0))
        q[:, b * BLOCK:(b + 1) * BLOCK] = _encode_blocks(part, s[:, b:b + 1].astype(np.int64))
    return q, s


def quantize_weights(W):
    W = np.asarray(W, dtype=np.float64)
    E, N, K = W.shape
    q = np.empty((E, N, K), np.uint8)
    s = np.full((E, -(-N // BLOCK), scale_cols(K)), 127, np.uint8)
    for e in range(E):
        for i in range(s.shape[1]):
            for j in range(-(-K // BLOCK)):
                sl = (e, slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                s[e, i, j] = scale_byte(np.abs(W[sl]).max())
                q[sl] = _encode_blocks(W[sl], np.int64(s[e, i, j]))
    return q, s


def dequantize_rows(q, s):
    C = q.shape[-1]
    return decode_e4m3(q) * np.repeat(decode_scale(s)[..., :-(-C // BLOCK)], BLOCK, axis=-1)[..., :C]


def dequantize_weights(q, s):
    E, N, K = q.shape
    return dequantize_rows(q, np.repeat(s, BLOCK, axis=1)[:, :N])


def round_bf16(v) -> np.ndarray:
    """Float64 values rounded to bf16 (8 significant bits, ties to even), as float64."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(v), np.round(v / step) * step, v)


def add_residual(x, residual):
    """r: the fp32 sum of two bf16 rows, rounded to bf16."""
    x = np.asarray(x, dtype=np.float32)
    if residual is not None:
        x = x + np.asarray(residual, dtype=np.float32)
    return round_bf16(x.astype(np.float64))


def norm(r, w, eps):
    """u before its rounding, and 1 / rms."""
    r, w = np.asarray(r, dtype=np.float64), np.asarray(w, dtype=np.float64)
    rstd = 1.0 / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    return r * rstd * w, rstd


def norm_backward(dy, dres, r, w, eps):
    """dx and dw before rounding."""
    dy, r, w = (np.asarray(v, dtype=np.float64) for v in (dy, r, w))
    _, rstd = norm(r, w, eps)
    c = (dy * w * r).mean(axis=1, keepdims=True)
    dx = rstd * w * dy - r * rstd ** 3 * c
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, (dy * r * rstd).sum(axis=0)


def grouped(a, W, offsets):
    """Rows offsets[e] .. offsets[e+1] of a [R, K] times W[e] [N, K]^T; NaN marks rows of no group."""
    out = np.full((a.shape[0], W.shape[1]), np.nan)
    for e in range(W.shape[0]):
        out[offsets[e]:offsets[e + 1]] = a[offsets[e]:offsets[e + 1]] @ W[e].T
    return out


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))
