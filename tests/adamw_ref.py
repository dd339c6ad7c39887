"""AdamW in 64 bits from its definition (numpy), and the 8-bit moments' codes, for the tests.

Shares nothing with the kernels: codes are looked up in tables written from their definition, and
rounding works on values, not on bit patterns."""
import numpy as np

E4M3 = np.array([np.nan if c & 127 == 127 else (-1.0) ** (c >> 7) * (
    (c & 7) / 8 * 2.0 ** -6 if c & 0x78 == 0 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])
ROOT = np.array([0.0] + [(1 + (c & 15) / 16) * 2.0 ** ((c >> 4) - 15) for c in range(1, 256)])


def blocks(x):
    """[ceil(n / 32), 32], zero-filled."""
    out = np.zeros((-(-x.size // 32), 32), x.dtype)
    out.reshape(-1)[:x.size] = x
    return out


def decode(codes, scales, table):
    v = table[codes.astype(np.int64)]
    s = np.where(scales == 0, 0.0, np.exp2(scales.astype(np.float64) - 127))
    s = np.where(scales == 255, np.nan, s)
    return v * np.repeat(s, 32)[:codes.size]


def mix(x):
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = x * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0x85EBCA77) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(13))


def random_bits(pos, seed, t):
    """16 bits each for m, r and a bf16 parameter at the given positions."""
    pos = np.asarray(pos, np.uint64)
    hi = pos >> np.uint64(32)
    base = np.uint64(int(mix((seed + 0x9E3779B9 * t) & 0xFFFFFFFF)) ^ (t >> 32))
    key = mix(base + hi)
    x = mix((pos & np.uint64(0xFFFFFFFF)) ^ key)
    y = ((x ^ (x >> np.uint64(7))) * np.uint64(0xC2B2AE3D)) & np.uint64(0xFFFFFFFF)
    return (x >> np.uint64(16)).astype(np.int64), (x & np.uint64(0xFFFF)).astype(np.int64), (y >> np.uint64(16)).astype(np.int64)


def step(p, g, m, v, t, lr, b1, b2, eps, wd, scale=1.0):
    """One step in 64 bits: (p, m, v)."""
    g = g.astype(np.float64) * scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p, m, v


def grid(x, top, mantissa, low):
    """x >= 0 in blocks of 32 -> (number of code steps of x under its block's scale, one step, scale
    exponent); a step is constant below 2^low."""
    b = blocks(x)
    amax = b.max(1, keepdims=True)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(amax / top)), -127)
        y = b / np.exp2(e)
        ulp = np.exp2(np.maximum(np.floor(np.log2(np.where(y > 0, y, 2.0 ** low))), low) - mantissa)
    n = x.size
    return (y / ulp).reshape(-1)[:n], (ulp * np.exp2(e)).reshape(-1)[:n], e.reshape(-1)
