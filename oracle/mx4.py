"""The 4-bit microscaled format in plain numpy (fp64): test infrastructure, no
code shared with the CUDA path.

A matrix is (codes [r, k] ints 0..15, scale bytes [r, k/32]); `pack` gives the
stored layout (two codes per byte, scale rows padded to 16 bytes).
"""
import numpy as np

MAGNITUDE = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rotate(x, signs=None):
    """x .* signs times the normalised 128-point Hadamard matrix per 128 columns."""
    x = np.asarray(x, dtype=np.float64)
    if signs is not None:
        x = x * np.asarray(signs, dtype=np.float64)
    h = np.array([[1.0]])
    while h.shape[0] < 128:
        h = np.block([[h, h], [h, -h]])
    return (x.reshape(-1, 128) @ h / np.sqrt(128.0)).reshape(x.shape)


def quantize(v):
    """Codes and scale bytes of finite or non-finite values, by the definition:
    the nearest magnitude, of two equally near ones that with the even code."""
    v = np.asarray(v, dtype=np.float64)
    r, k = v.shape
    codes = np.zeros((r, k), dtype=np.uint8)
    scales = np.zeros((r, k // 32), dtype=np.uint8)
    for i in range(r):
        for b in range(k // 32):
            block = v[i, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(block)):
                scales[i, b] = 255
                continue
            top = np.abs(block).max()
            e = -127 if top == 0 else max(-127, min(127, int(np.frexp(top)[1]) - 1 - 2))
            scales[i, b] = e + 127
            a = np.abs(np.ldexp(block, -e))
            d = np.abs(a[:, None] - MAGNITUDE[None, :])
            near = d == d.min(axis=1, keepdims=True)
            first = near.argmax(axis=1)
            last = 7 - near[:, ::-1].argmax(axis=1)
            codes[i, 32 * b:32 * b + 32] = np.where(first % 2 == 0, first, last) + 8 * np.signbit(block)
    return codes, scales


def values(codes, scales):
    """fp64 values of codes and scale bytes (byte 255: NaN)."""
    codes = np.asarray(codes)
    m = MAGNITUDE[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127)
    s = np.where(np.asarray(scales) == 255, np.nan, s)
    return m * np.repeat(s, 32, axis=-1)


def stride(k):
    return (k + 511) // 512 * 16


def pack(codes, scales):
    codes = np.asarray(codes, dtype=np.uint8)
    padded = np.zeros(codes.shape[:-1] + (stride(codes.shape[-1]),), dtype=np.uint8)
    padded[..., :scales.shape[-1]] = scales
    return codes[..., 0::2] | (codes[..., 1::2] << 4), padded


def unpack(packed, padded):
    packed = np.asarray(packed)
    codes = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), dtype=np.uint8)
    codes[..., 0::2], codes[..., 1::2] = packed & 15, packed >> 4
    return codes, np.asarray(padded)[..., :codes.shape[-1] // 32]
