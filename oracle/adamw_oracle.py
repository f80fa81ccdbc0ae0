"""Float64 AdamW, its 8-bit moments, and the global gradient norm (numpy).

Used by the tests only.  Moments in 8 bits: blocks of 256 elements of one
tensor, m as e4m3 times (largest |m| / 256), v as an unsigned 5-exponent,
3-mantissa-bit float times the block's largest v.
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
M_NAN, V_NAN = 0x7F, 255


def moments(m, v, g, beta1, beta2, scale=1.0):
    y = np.asarray(g, np.float64) * scale
    return (beta1 * np.asarray(m, np.float64) + (1 - beta1) * y,
            beta2 * np.asarray(v, np.float64) + (1 - beta2) * y * y)


def update(w, m, v, t, lr, beta1, beta2, eps, lr_scale=1.0, weight_decay=0.0):
    """w_t from w_{t-1} and the new moments."""
    w = np.asarray(w, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        adam = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w - lr * (lr_scale * adam + weight_decay * w)


# ---------------------------------------------------------------------------
# Rounding bits
# ---------------------------------------------------------------------------
def mix(x):
    """The counter hash's mixing of 32-bit values (uint64 arrays, products modulo 2^32)."""
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def key(seed: int, t: int) -> int:
    k = int(mix((t >> 32) ^ 0x3C6EF372))
    k = int(mix((t & 0xFFFFFFFF) ^ k))
    k = int(mix((seed >> 32) ^ k))
    return int(mix((seed & 0xFFFFFFFF) ^ k))


def random_bits(index, seed: int, t: int):
    """(bits of m, bits of v), 16 each, of the elements with these indexes in the batch."""
    index = np.asarray(index, np.uint64)
    lo, hi = index & np.uint64(0xFFFFFFFF), index >> np.uint64(32)
    h = mix(lo + mix(np.uint64(key(seed, t)) + hi))
    return h & np.uint64(0xFFFF), h >> np.uint64(16)


# ---------------------------------------------------------------------------
# Codes
# ---------------------------------------------------------------------------
def _blocks(x):
    pad = -len(x) % BLOCK
    return np.pad(x, (0, pad)).reshape(-1, BLOCK)


def scales(m, v):
    """(m_scale, v_scale) of every block, over its finite elements."""
    m, v = np.asarray(m, np.float64), np.asarray(v, np.float64)
    am = np.where(np.isfinite(m), np.abs(m), 0.0)
    av = np.where(np.isfinite(v) & (v > 0), v, 0.0)
    top = _blocks(am).max(axis=1)
    return np.where(top >= 2.0 ** -118, top / 256, 0.0), _blocks(av).max(axis=1)


def _spread(scale, n):
    return np.repeat(scale, BLOCK)[:n]


def positions(x, scale, low):
    """(position in code steps, step) of |x| / scale; steps below 2^low stay those of [2^low, 2^(low+1))."""
    s = _spread(scale, len(x))
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(np.where(np.isfinite(x), x, 0.0)) / s, 0.0)
    e = np.maximum(np.frexp(y)[1] - 1, low)
    step = np.ldexp(1.0, e - 3)
    return y / step, step


def decode_m(code, scale):
    code = np.asarray(code, np.int64)
    e, f = (code >> 3) & 15, code & 7
    y = np.where(e > 0, np.ldexp(1 + f / 8, e - 7), np.ldexp(f / 8, -6))
    y = np.where((code & 0x7F) == 0x7F, np.nan, np.where(code & 0x80, -y, y))
    return y * _spread(scale, len(code))


def decode_v(code, scale):
    code = np.asarray(code, np.int64)
    y = np.where(code == 0, 0.0, np.ldexp(1 + (code & 7) / 8, (code >> 3) - 31))
    return np.where(code == V_NAN, np.nan, y) * _spread(scale, len(code))


def encode_m(m, scale, up):
    """Codes of m; `up` in (0, 1) is what rounding adds before the cut (1/2: nearest)."""
    m = np.asarray(m, np.float64)
    pos, step = positions(m, scale, -6)
    y = np.minimum(np.floor(pos + up) * step, 448.0)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    f = y / np.ldexp(1.0, e)              # in [0, 2): below 1 only in the subnormal range
    code = np.where(f >= 1, (e + 7) * 8 + (f - 1) * 8, f * 8).astype(np.int64)
    code = code | np.where(np.signbit(m), 0x80, 0)
    return np.where(np.isfinite(m), code, M_NAN).astype(np.uint8)


def encode_v(v, scale, up):
    v = np.asarray(v, np.float64)
    pos, step = positions(v, scale, -31)
    y = np.minimum(np.floor(pos + up) * step, 1.0)
    y = np.maximum(y, 1.125 * 2.0 ** -31)
    e = np.frexp(y)[1] - 1
    code = ((e + 31) * 8 + (y / np.ldexp(1.0, e) - 1) * 8).astype(np.int64)
    code = np.where(v > 0, code, 0)
    return np.where(np.isfinite(v) & (v >= 0), code, V_NAN).astype(np.uint8)


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------
def grad_norm(grads, max_norm):
    """(N, coefficient, every tensor's norm)."""
    sq = [float(np.sum(np.square(np.asarray(g, np.float64).ravel()))) for g in grads]
    norm = float(np.sqrt(np.sum(sq)))
    coef = 1.0 if norm <= max_norm else max_norm / norm
    return norm, coef, np.sqrt(sq)
