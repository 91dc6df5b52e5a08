"""Plain 64-bit forms of the paged-cache operators and of draft verification (numpy, one sequence
and one token at a time, straight from the definitions in include/kda.h), and the bounds that the
kernels' roundings allow."""
import numpy as np

U32, STEP = 2.0 ** -24, {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}


def visible(length, m, j, window):
    hi = length - m + 1 + j
    return (max(0, hi - window) if window else 0), hi


def attend(q, k, v, page_ok, lens, scale, window):
    """q [N, m, Hq, d]; k, v: per sequence [len, Hkv, d]; page_ok: per sequence bool [len].
    Returns o [N, m, Hq, d] and lse [N, m, Hq]."""
    N, m, Hq, d = q.shape
    o = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for n in range(N):
        G = Hq // k[n].shape[1]
        for j in range(m):
            lo, hi = visible(lens[n], m, j, window)
            at = [t for t in range(lo, max(lo, hi)) if page_ok[n][t]]
            if not at:
                continue
            for h in range(Hq):
                s = scale * (k[n][at, h // G] @ q[n, j, h])
                top = s.max()
                w = np.exp(s - top)
                o[n, j, h] = (w / w.sum()) @ v[n][at, h // G]
                lse[n, j, h] = top + np.log(w.sum())
    return o, lse


def attend_bound(q, k, v, lens, scale, cache, ref, out):
    """How far an output may be off. A score is a dot product of d terms in 32 bits, scaled
    (d + 3 roundings of at most scale |q| |k|); a weight takes it absolutely, and once more through
    the sum that divides it; 2^x is good to one unit in 2^-23 (twice); the sum and the product
    with V take one rounding for each 16 tokens of a wave's share, at most L / 16 + 64. bf16 and
    e4m3 caches round each weight to 16 bits (2^-17). Then the result is rounded to its type."""
    d = q.shape[-1]
    L = max([1] + [int(x) for x in lens])
    kn = max([0.0] + [np.sqrt((x.astype(np.float64) ** 2).sum(-1)).max() for x in k if x.size])
    vm = max([0.0] + [np.abs(x).max() for x in v if x.size])
    qn = np.sqrt((q.astype(np.float64) ** 2).sum(-1)).max()
    e = 2 * (d + 3) * U32 * abs(scale) * qn * kn + 4 * 2.0 ** -23 + 2 * (L / 16 + 64) * U32
    e += 0.0 if cache == "f32" else 2 * 2.0 ** -17
    return vm * e * 1.01 + STEP[out] * np.abs(ref)


def rotate(x, pos, inv_freq, pairs):
    """x [heads, d] at a position; the angle in 64 bits."""
    y = x.astype(np.float64).copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        t = float(pos) * float(inv_freq[i])
        c, s = np.cos(t), np.sin(t)
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


def verify(p, q, x, r, counts):
    """p [N, m + 1, V], q [N, m, V] or None, x [N, m], r [N, m + 1]: (accept, tokens)."""
    N, m = x.shape
    V = p.shape[2]
    top = np.nextafter(np.float32(1), np.float32(0))
    accept, tokens = [], []
    for n in range(N):
        u = [float(min(max(z, 0.0), top)) if z == z else 0.0 for z in r[n].astype(np.float64)]
        c = min(max(int(counts[n]), 0), m)
        a = 0
        while a < c and 0 <= x[n, a] < V:
            px = float(p[n, a, x[n, a]])
            qx = 1.0 if q is None else float(q[n, a, x[n, a]])
            if not (np.isfinite(px) and np.isfinite(qx) and u[a] * qx < px):
                break
            a += 1
        clean = lambda z: np.where(np.isfinite(z) & (z > 0), z, 0).astype(np.float64)  # noqa: E731
        w = full = clean(p[n, a])
        if a < c:
            if q is not None:
                w = np.maximum(full - clean(q[n, a]), 0)
            else:
                w = full.copy()
                if 0 <= x[n, a] < V:
                    w[x[n, a]] = max(w[x[n, a]] - 1.0, 0.0)
        if not w.sum() > 0:
            w = full
        nxt = -1
        if w.sum() > 0:
            cum = np.cumsum(w)
            past = np.nonzero(cum > u[m] * cum[-1])[0]
            nxt = int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])
        accept.append(a)
        tokens.append(list(x[n, :a]) + [nxt] + [-1] * (m - a))
    return np.array(accept), np.array(tokens)
