"""Rotary positions from their definition, in float64 on the host, and bf16 rows."""
import math

import numpy as np

from paged_kv_cache_pg_gb300 import pkv


def bf16_bits(x):
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def random_rows(rng, *shape):
    return bf16_bits(rng.standard_normal(shape))


def freqs(rot, base, scaling="plain", factor=1.0, original=0, fast=None, slow=None):
    """(radians a position of each pair, scale)."""
    out, scale = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "ntk":
            f = (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif scaling == "yarn":
            at = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            low, high = max(0, math.floor(at(fast or 32))), min(rot - 1, math.ceil(at(slow or 1)))
            part = min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
            f, scale = f / factor * part + f * (1 - part), 0.1 * math.log(factor) + 1
        elif scaling == "bands":
            n = original * f / (2 * math.pi)
            hi, lo = fast or 4.0, slow or 1.0
            f = f if n >= hi else f / factor if n <= lo else f / factor + (f - f / factor) * (n - lo) / (hi - lo)
        out.append(f)
    return np.array(out), scale


def turn(x, pos, rot, pairs, f, scale):
    """x float64 [tokens][heads][dim], pos [tokens] -> (rotated, |a| + |b| of each element's pair)."""
    angle = np.asarray(pos, np.float64)[:, None] * f
    c, s = (t(angle)[:, None] * scale for t in (np.cos, np.sin))
    y, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == pkv.ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size * abs(scale)


def slack(size):
    """What float32 may add to an element: cosine and sine each within 2^-23 of a unit for their angle
    (a 32-bit fraction of a turn, rounded to 24 bits: pi 2^-25) and 2^-23 for the function and the
    scale, two products and a sum of 2^-24 each: 2^-21 of |a| + |b| holds it twice over."""
    return size * 2.0 ** -21
