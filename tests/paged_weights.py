"""Attention rows that see two tokens, whose results show how many bits the softmax weights were
held in: the first token has score 0 and value 0, the second score s < 0 and value v, so that
o = v w / (1 + w) with w = e^s, and an error of w is one of o."""
import numpy as np

U = 2.0 ** -24


def make(seed, cache, N, Hq, Hkv, d):
    """q [N, 1, Hq, d]; k, v [N, 2, Hkv, d] (values that bf16 and e4m3 hold), scales [2, Hkv], scale."""
    rng = np.random.default_rng(seed)
    q, k, v = np.zeros((N, 1, Hq, d)), np.zeros((N, 2, Hkv, d)), np.zeros((N, 2, Hkv, d))
    q[..., 0] = rng.integers(64, 256, (N, 1, Hq)) / 128  # 8 bits, 0.5 .. 2
    k[:, 1, :, 0] = -rng.integers(8, 16, (N, Hkv)) / rng.choice([16, 8, 4, 2], (N, Hkv))  # 4 bits
    v[:, 1] = rng.integers(8, 16, (N, Hkv, d)) / 8 * rng.choice([-1, 1], (N, Hkv, d))
    scales = np.ones((2, Hkv), np.float32)
    if cache == "e4m3":
        scales = np.exp(rng.uniform(-0.3, 0.3, (2, Hkv))).astype(np.float32)
    return q, k, v, scales, float(np.float32(0.115))


def reference(q, k, v, scales, scale, weight=lambda w: w):
    """o [N, Hq, d] and s [N, Hq] in 64 bits; `weight` rounds the second token's weight."""
    G = q.shape[2] // k.shape[2]
    up = lambda x: np.repeat(x, G, axis=1)  # noqa: E731
    s = scale * q[:, 0, :, 0] * up(k[:, 1, :, 0] * scales[0].astype(np.float64))
    w = np.exp(s)
    o = (weight(w) / (1 + w))[..., None] * up(v[:, 1] * scales[1].astype(np.float64)[:, None])
    return o, s


def relative_bound(s, cache):
    """How far o may be off before it is rounded to its type, relative to it, with every weight held
    to 24 bits, counted in units of 2^-24:
      6 |s|  the score's constant, its three factors and its dot product (the last may be cut off: 2)
      4      2^x, one unit in 2^-23, for w and for the first token's weight
      6      the weight's parts added up in the matrix product, at most three, each cut off
      4      the sum of weights and that of the products, within a wave and over the waves
      2      v_scale over the sum, and its product
    over e4m3 the exponent is raised by 14 (below 16 in size: 2^-21 of log2, 5.6) and two fp16 parts
    hold 22 bits and a sign (2)."""
    return (6 * np.abs(s) + 16 + (7.6 if cache == "e4m3" else 0.0)) * U


def to_bf16(x):
    """Rounded to nearest even, as float64."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return b.view(np.float32).astype(np.float64)


def outside(got, o, s, cache, out):
    """Number of results that lie outside what the bound allows."""
    e = relative_bound(s, cache)[..., None] * np.abs(o)
    lo, hi = o - e, o + e
    if out == "bf16":
        lo, hi = to_bf16(lo), to_bf16(hi)
    else:
        lo, hi = lo - U * np.abs(o), hi + U * np.abs(o)
    return int(((got < lo) | (got > hi)).sum())
