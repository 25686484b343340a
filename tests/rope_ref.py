"""The rotation by position from its definition (include/dqmoe.h, dq_kv_append_rope) in numpy and 64 bits."""
import numpy as np


def pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, pos, inv_freq, interleaved=False, factor=1.0):
    """x [T][H][D] -> (the rotated rows, |a| + |b| of every value's pair: 0 where nothing turns)."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    angle = np.asarray(pos, dtype=np.float64)[:, None] * f
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    one, two = pairs(2 * len(f), interleaved)
    a, b = x[..., one], x[..., two]
    y, size = x.copy(), np.zeros_like(x)
    k = float(np.float32(factor))
    y[..., one], y[..., two] = (a * c - b * s) * k, (b * c + a * s) * k
    size[..., one] = size[..., two] = (np.abs(a) + np.abs(b)) * k
    return y, size


def frequencies(R, base=10000.0):
    return (base ** (-np.arange(0, R, 2) / R)).astype(np.float32)


def quantise(x):
    """x [..., D] in 64 bits -> (codes, scales [..., D / 32]) of Q4_0 blocks: exact arithmetic, but that the scale is
    the fp16 nearest to -1/8 of the largest value's fp32."""
    g = np.clip(np.asarray(x, dtype=np.float64), -65504.0, 65504.0).reshape(*x.shape[:-1], -1, 32)
    m = np.take_along_axis(g, np.argmax(np.abs(g), axis=-1)[..., None], -1)
    d = (m.astype(np.float32) / np.float32(-8)).astype(np.float16).astype(np.float64)
    c = np.clip(np.floor(g / np.where(d == 0, 1.0, d) + 8.5), 0, 15)
    return np.where(d == 0, 8, c).astype(np.int64).reshape(x.shape), d[..., 0]
