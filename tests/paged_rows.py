"""Attention over what each row sees, with a bound for each result from that row's own weights, scores
and values (64 bits, numpy)."""
import numpy as np

from tests.paged_ref import visible
from tests.paged_weights import U, to_bf16


def attend_rows(q, k, v, lens, scale, window, cache, weight=lambda w: w):
    """q [N, m, Hq, d]; k, v: per sequence [len, Hkv, d], scales included. Returns o and what it may be
    off by before it is rounded to its type (of o's shape), lse and what it may be off by. `weight`
    rounds the weights 2^{(s - max) / ln 2}.

    The bound, with u = 2^-24 and A_t = scale sum_c |q_c k_tc|:
      a score is off by (2 d + 8) u A_t (d additions in the matrix product that may cut off, the constant
      and the factors), and by u times the exponent it enters, x_t = (max - s_t) / ln 2, plus the 14 by
      which it is raised over e4m3; a weight takes that relatively, and again through the sum that
      divides it;
      a tile of 32 tokens adds at most 48 u: 10 additions to the sum of weights, 34 in the matrix product
      (three bf16 parts of 8 each, or 8 fp32 instructions of 4 products and one rounding), 4 where the
      maximum moves; the tiles of a row are those of its tokens, and at most one more for each of
      four waves and their joins (8);
      2^x is good to one unit in 2^-23, v_scale, the division, two fp16 parts: 16 u."""
    N, m, Hq, d = q.shape
    o, off = np.zeros(q.shape), np.zeros(q.shape)
    lse, lse_off = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for n in range(N):
        H = k[n].shape[1]
        G = Hq // H
        for j in range(m):
            lo, hi = visible(lens[n], m, j, window)
            if hi <= lo:
                continue
            kk, vv = k[n][lo:hi].transpose(1, 0, 2), v[n][lo:hi].transpose(1, 0, 2)  # [H, t, d]
            qq = q[n, j].reshape(H, G, d)
            s = scale * (qq @ kk.transpose(0, 2, 1))
            A = abs(scale) * (np.abs(qq) @ np.abs(kk).transpose(0, 2, 1))
            top = s.max(-1, keepdims=True)
            w = weight(np.exp(s - top))
            full = np.exp(s - top)
            p = w / full.sum(-1, keepdims=True)
            rel = ((2 * d + 8) * A + (top - s) / np.log(2.0) + (14 if cache == "e4m3" else 0)).max(-1, keepdims=True)
            tiles = (hi - lo + 31) // 32 + 8
            o[n, j] = (p @ vv).reshape(Hq, d)
            off[n, j] = ((p @ np.abs(vv)) * (2 * rel + 48 * tiles + 16) * U).reshape(Hq, d)
            lse[n, j] = (top[..., 0] + np.log(full.sum(-1))).reshape(Hq)
            # log2 to one unit, its product and the sum with the maximum
            lse_off[n, j] = ((rel + 48 * tiles + 16)[..., 0] * U).reshape(Hq) + 8 * U * (1 + np.abs(lse[n, j]))
    return o, off, lse, lse_off


def outside(got, o, off, out):
    """Where results lie outside what the bound allows."""
    lo, hi = o - off, o + off
    if out == "bf16":
        lo, hi = to_bf16(lo), to_bf16(hi)
    else:
        lo, hi = lo - U * np.abs(o), hi + U * np.abs(o)
    return ~((got >= lo) & (got <= hi))
