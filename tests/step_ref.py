"""Plain 64-bit forms of linear attention with a decay per head, of page plans and of adjusted logits,
straight from the definitions in kda.h: one token, one sequence, one row after the other."""
import numpy as np


def lin(q, k, v, g, S0, scale, lengths=None):
    """q, k [T, Hk, dk], v [T, H, dv], g [T, H] or [H], of packed sequences (lengths, default one);
    S0 [n_seq, H, dk, dv] or None. Returns o [T, H, dv], S_T, and for each of them the same sums over
    absolute values, which rounding errors are relative to."""
    q, k, v, g = (np.asarray(x, np.float64) for x in (q, k, v, g))
    T, H, dv = v.shape
    rep, dk = H // q.shape[1], q.shape[2]
    q, k = q.repeat(rep, 1), k.repeat(rep, 1)
    g = np.broadcast_to(g, (T, H))
    lengths = [T] if lengths is None else lengths
    S = np.zeros((len(lengths), H, dk, dv)) if S0 is None else np.array(S0, np.float64)
    A = np.abs(S)
    o, ao = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    t = 0
    for n, length in enumerate(lengths):
        for _ in range(length):
            a = np.exp(g[t])[:, None, None]
            S[n] = a * S[n] + k[t][:, :, None] * v[t][:, None, :]
            A[n] = a * A[n] + np.abs(k[t][:, :, None] * v[t][:, None, :])
            o[t] = scale * np.einsum("hk,hkv->hv", q[t], S[n])
            ao[t] = abs(scale) * np.einsum("hk,hkv->hv", np.abs(q[t]), A[n])
            t += 1
    return o, S, ao, A


def plan(table, held, lens, new_lens, free, ring, page_size, max_tokens):
    """Everything that page_plan returns or changes, as a dict; its arguments stay."""
    table, free = table.copy(), free.copy()
    N, width = table.shape
    cap = len(free)
    before = free.copy()
    head, count = max(int(ring[0]), 0) % cap, min(max(int(ring[1]), 0), cap)
    held = [min(max(int(x), 0), width) for x in held]
    lens = [max(int(x), 0) for x in lens]
    seq, cu, slots, positions = [], [0], [], []
    asked = asked_tokens = used = given = 0
    for n in range(N):
        new = int(new_lens[n])
        if new < 0:
            for p in range(held[n]):
                if count + given < cap:
                    free[(head + count + given) % cap] = table[n, p]
                    given += 1
            held[n] = 0
            seq.append(0)
            cu.append(cu[-1])
            continue
        pages = -(-(lens[n] + new) // page_size)
        ok = pages <= width and lens[n] + new < 2 ** 31
        if ok:
            need = max(0, pages - held[n])
            asked += need
            asked_tokens += new
            ok = (need == 0 or asked <= count) and (new == 0 or asked_tokens <= max_tokens)
        if ok:
            for _ in range(need):
                table[n, held[n]] = before[(head + used) % cap]
                held[n] += 1
                used += 1
            for pos in range(lens[n], lens[n] + new):
                page = int(table[n, pos // page_size])
                slots.append(-1 if page < 0 else page * page_size + pos % page_size)
                positions.append(pos)
        seq.append(lens[n] + (new if ok else 0))
        cu.append(cu[-1] + (new if ok else 0))
    rest = [-1] * (max_tokens - cu[-1])
    return dict(table=table, free=free, held=np.array(held), ring=np.array([(head + used) % cap, count - used + given]),
                seq_lens=np.array(seq), cu=np.array(cu), slots=np.array(slots + rest),
                positions=np.array(positions + rest))


def logits(x, history=None, history_lens=None, prompt_lens=None, drafts=None, repetition=None, frequency=None,
           presence=None, bias_ids=None, bias=None, bias_counts=None, mask=None, temperature=None, probs=False):
    """Adjusted logits or probabilities of x [N, R, V], in 64 bits."""
    x = np.array(x, np.float64)
    N, R, V = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        for n in range(N):
            ids = []
            prompt = 0
            if history is not None:
                length = min(max(int(history_lens[n]), 0), history.shape[1])
                ids = [int(i) for i in history[n, :length]]
                prompt = min(max(int(prompt_lens[n]), 0), length) if prompt_lens is not None else 0
            for j in range(R):
                y = x[n, j]
                said = ids[prompt:] + ([int(i) for i in drafts[n, :j]] if drafts is not None else [])
                said = [i for i in said if 0 <= i < V]
                there = set(said) | {i for i in ids[:prompt] if 0 <= i < V}
                r = 1.0 if repetition is None else float(repetition[n])
                f = 0.0 if frequency is None else float(frequency[n])
                p = 0.0 if presence is None else float(presence[n])
                for i in there:
                    y[i] = y[i] / r if y[i] > 0 else y[i] * r
                for i in set(said):
                    y[i] -= f * said.count(i) + p
                if bias is not None:
                    count = bias.shape[1] if bias_counts is None else min(max(int(bias_counts[n]), 0), bias.shape[1])
                    last = {int(bias_ids[n, e]): float(bias[n, e]) for e in range(count)}
                    for i, b in last.items():
                        if 0 <= i < V:
                            y[i] += b
                if mask is not None:
                    words = np.asarray(mask[n, j]).astype(np.int64) & 0xffffffff
                    i = np.arange(V)
                    y[(words[i // 32] >> (i % 32)) & 1 == 0] = -np.inf
                t = 1.0 if temperature is None else float(temperature[n])
                greedy = not t > 0
                if not greedy:
                    y /= t
                if probs:
                    x[n, j] = pick(y) if greedy else softmax(y)
    return x


def pick(y):
    p = np.zeros_like(y)
    z = np.where(np.isnan(y), -np.inf, y)
    if z.max() > -np.inf:
        p[int(np.argmax(z))] = 1.0
    return p


def softmax(y):
    if np.isnan(y).any():
        return np.full_like(y, np.nan)
    top = y.max()
    if top == -np.inf:
        return np.zeros_like(y)
    e = (y == np.inf).astype(np.float64) if top == np.inf else np.exp(y - top)
    return e / e.sum()
