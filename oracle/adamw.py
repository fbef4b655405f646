"""Oracle: the AdamW step, in fp64 and (``step_f32``) in fp32 with one rounding
per operation, and the 8-bit moments' codes.

The pages name no optimizer; this is the published rule with decoupled weight
decay.  8-bit moments: blocks of 256 elements share an fp32 scale; the first
moment is E4M3 times max |m| * fp32(1 / 448), the second an unsigned float with 3
mantissa bits (code c stands for the fp32 with bits (c + 762) << 20, so 254 is
1.0, and 0 for zero, 255 for NaN) times max v; both rounded stochastically
with 16 bits of a hash of (seed, step, tensor, element)."""

import numpy as np

BLOCK = 256
M32 = 0xFFFFFFFF


def step_f64(p, g, m, v, t, lr, betas, eps, wd):
    """New parameter and moments, and the update with the magnitudes of the
    first moment's two terms in place of their sum (>= |update|: what its
    roundings are relative to, the terms may cancel)."""
    b1, b2 = betas
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    mag = np.abs(b1 * m) + np.abs((1 - b1) * g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    rate = lr / (1 - b1 ** t) / (np.sqrt(v) / np.sqrt(1 - b2 ** t) + eps)
    return p * (1 - lr * wd) - rate * m, m, v, rate * mag


def moments_f32(g, m, v, betas, grad_scale=1.0):
    """The new moments exactly as the fp32 definition rounds them."""
    f = np.float32
    b1, c1, b2, c2 = f(betas[0]), f(1 - betas[0]), f(betas[1]), f(1 - betas[1])
    with np.errstate(over="ignore", invalid="ignore"):
        g = np.asarray(g, f) * f(grad_scale)
        return b1 * np.asarray(m, f) + c1 * g, b2 * np.asarray(v, f) + c2 * (g * g)


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & M32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & M32
    return x ^ (x >> 16)


def random_bits(seed, step, tensor, n):
    key = _mix((_mix((_mix(seed & M32) + step) & M32) + tensor) & M32)
    i = np.arange(n, dtype=np.uint64)
    m = np.uint64(M32)
    x = ((i * np.uint64(0x9E3779B1)) & m) ^ np.uint64(key) ^ (((i >> np.uint64(32)) * np.uint64(0x6A09E667)) & m)
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x9E3779B9)) & m
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xBB67AE85)) & m
    return (x ^ (x >> np.uint64(16))).astype(np.uint32)


def _blocks(x):
    n = x.size
    return np.concatenate([x, np.zeros(-n % BLOCK, x.dtype)]).reshape(-1, BLOCK)


def _per_element(s, n):
    return np.repeat(s, BLOCK)[:n]


def encode(m, v, r):
    """(m codes, m scales, v codes, v scales) of fp32 moments with random
    bits r (uint32 per element)."""
    f = np.float32
    m, v = np.asarray(m, f), np.asarray(v, f)
    n = m.size
    ms = (np.abs(_blocks(np.where(np.isfinite(m), m, f(0)))).max(axis=1) * (f(1) / f(448))).astype(f)
    vs = _blocks(np.where(np.isfinite(v), v, f(0))).max(axis=1).astype(f)
    with np.errstate(all="ignore"):
        s = _per_element(ms, n)
        y = np.minimum(np.abs(m) / s, f(448)).astype(f)
        rm = (r >> np.uint32(16)).astype(np.uint32)
        low = np.floor(y * f(512) + rm.astype(f) / f(65536))
        high = ((y.view(np.uint32).astype(np.int64) + (rm.astype(np.int64) << 4)) >> 20) - (120 << 3)
        mc = np.where(y < f(2.0 ** -6), np.nan_to_num(low).astype(np.int64), high)
        mc = np.where(s > 0, mc, 0)
        mc = np.where(np.isfinite(m), mc, 0x7F) | np.where(np.signbit(m), 0x80, 0)
        s = _per_element(vs, n)
        y = (v / s).astype(f)
        rv = (r & np.uint32(0xFFFF)).astype(np.int64)
        vc = np.clip(((y.view(np.uint32).astype(np.int64) + (rv << 4)) >> 20) - 762, 1, 254)
        vc = np.where(v > 0, vc, 0)    # (a quotient that underflows takes the lowest code)
        vc = np.where(np.isfinite(v), vc, 255)
    return mc.astype(np.uint8), ms, vc.astype(np.uint8), vs


def decode(mc, ms, vc, vs):
    from .nvfp4 import e4m3_decode
    f = np.float32
    n = mc.size
    mag = e4m3_decode((np.where((mc & 0x7F) == 0x7F, 0, mc) & 0x7F).astype(np.uint8)).astype(f)
    m = np.where(mc & 0x80, -mag, mag).astype(f) * _per_element(ms, n)
    m = np.where((mc & 0x7F) == 0x7F, f(np.nan), m)
    x = ((vc.astype(np.uint32) + np.uint32(762)) << np.uint32(20)).view(f)
    v = np.where(vc > 0, x, f(0)) * _per_element(vs, n)
    return m.astype(f), np.where(vc == 255, f(np.nan), v).astype(f)
