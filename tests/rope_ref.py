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
