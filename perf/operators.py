"""Cases of the serving operators that stand next to the KDA kernels: appending keys and values to
a paged cache, attention of new tokens over that cache, and the verification of drafted tokens.

Each case is one operator call of a serving step. `run` computes it with elementary torch
operations, or, where `own` is true, with this package's operators.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}
DEV = "cuda"


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one conversation at its start: the latency of a single short call
        dict(name="attn-one", op="attn", N=1, m=1, Hq=32, Hkv=8, d=128, lo=300, hi=300, page=16,
             window=0, cache="bf16", idle=0),
        # sixteen requests whose contexts differ widely (the lengths of the varlen-16 workload)
        dict(name="attn-varlen-16", op="attn", N=16, m=1, Hq=32, Hkv=8, d=128, lo=512, hi=16384,
             page=64, window=0, cache="bf16", idle=0),
        # a full serving batch (decode-512) verifying four drafts on an 8-bit cache, some slots idle
        dict(name="attn-512-drafts-e4m3", op="attn", N=512, m=4, Hq=32, Hkv=8, d=128, lo=5, hi=4096,
             page=32, window=0, cache="e4m3", idle=37),
        # few very long contexts
        dict(name="attn-64k", op="attn", N=4, m=1, Hq=64, Hkv=8, d=128, lo=61001, hi=65536,
             page=256, window=0, cache="bf16", idle=0),
        # fp32 model with small heads, an odd group, a window and pages that end inside tiles
        dict(name="attn-window-f32", op="attn", N=12, m=3, Hq=6, Hkv=2, d=64, lo=1, hi=5003,
             page=48, window=1000, cache="f32", idle=0),
        # one new token of each of 512 sequences: a decode step's append
        dict(name="append-512", op="append", B=512, T=1, packed=0, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, lo=5, hi=131071, page=64, act="bf16", cache="bf16"),
        # sixteen packed prompts, 65,536 tokens: the append of a prefill
        dict(name="append-prompts", op="append", B=1, T=65536, packed=16, Hq=32, Hkv=8, d=128,
             rot=128, interleaved=False, lo=0, hi=4095, page=64, act="bf16", cache="bf16"),
        # four drafts of each of 64 sequences into an 8-bit cache, partial rotation by pairs
        dict(name="append-drafts-e4m3", op="append", B=64, T=4, packed=0, Hq=24, Hkv=4, d=64,
             rot=32, interleaved=True, lo=1, hi=70001, page=16, act="bf16", cache="e4m3"),
        # one request with four drafts: the latency of a single small call
        dict(name="verify-one", op="verify", N=1, m=4, V=32000, probs="f32", drawn=True,
             ragged=False),
        # a serving batch with a large vocabulary
        dict(name="verify-256", op="verify", N=256, m=4, V=131072, probs="f32", drawn=True,
             ragged=False),
        # bf16 probabilities, an odd vocabulary, and sequences with fewer drafts than others
        dict(name="verify-ragged-bf16", op="verify", N=48, m=8, V=50257, probs="bf16", drawn=True,
             ragged=True),
        # drafts that were picked (looked up, or by argmax) rather than drawn: no draft probabilities
        dict(name="verify-picked", op="verify", N=128, m=3, V=100003, probs="f32", drawn=False,
             ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "verify"])
    if op == "attn":
        N = _log(rng, 1, 300)
        most = min(65536, max(64, (1 << 18) // N))
        hi = _log(rng, 40, most)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, N=N, m=rng.choice([1, 1, 2, 3, 4, 5, 8]),
                    Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv,
                    d=rng.choice([32, 64, 128, 128]), lo=rng.randint(1, hi), hi=hi,
                    page=rng.choice([1, 8, 16, 20, 32, 48, 64, 128, 256]),
                    window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]),
                    cache=rng.choice(["bf16", "bf16", "e4m3", "f32"]),
                    idle=rng.choice([0, 0, 3, 11]))
    if op == "append":
        act = rng.choice(["bf16", "bf16", "f32"])
        packed = rng.choice([0, 0, _log(rng, 1, 40)])
        tokens = _log(rng, 1, 40000)
        T = max(tokens, packed) if packed else rng.choice([1, 1, 2, 4, 7, _log(rng, 1, 3000)])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([32, 64, 128, 128])
        return dict(op=op, B=1 if packed else max(1, tokens // T), T=T, packed=packed,
                    Hq=Hkv * rng.choice([1, 2, 4, 5]), Hkv=Hkv, d=d,
                    rot=rng.choice([0, 16, d // 2, d, d]), interleaved=rng.random() < 0.4,
                    lo=0, hi=_log(rng, 1, 100000), page=rng.choice([1, 8, 16, 20, 48, 64, 256]),
                    act=act, cache="f32" if act == "f32" else rng.choice(["bf16", "bf16", "e4m3"]))
    m = rng.choice([1, 2, 3, 4, 5, 8, 12])
    V = _log(rng, 7, 160001)
    return dict(op=op, N=min(_log(rng, 1, 300), max(1, (1 << 27) // (m * V))), m=m, V=V,
                probs=rng.choice(["f32", "f32", "bf16"]), drawn=rng.random() < 0.7,
                ragged=rng.random() < 0.4)


# --------------------------------------------------------------------------------- inputs

def _lengths(c):
    """Cached lengths of a case: spread evenly from lo to hi; `idle` of them are empty slots."""
    n = c["N"]
    full = [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) for i in range(n)]
    full[0] = c["hi"]
    for i in range(min(c["idle"], n - 1)):
        full[1 + i * (n - 1) // c["idle"]] = 0
    return full


def _pages(lengths, page, gen):
    """A block table whose sequences own pages of a shuffled pool, and the pool's size."""
    used = [-(-x // page) for x in lengths]
    width = max(1, max(used))
    have = torch.tensor(used)
    mine = torch.arange(width)[None, :] < have[:, None]
    pool = sum(used) + 3
    table = torch.full((len(lengths), width), -1, dtype=torch.int64, device=DEV)
    table[mine.to(DEV)] = torch.randperm(pool, generator=gen, device=DEV)[:sum(used)]
    return table.to(torch.int32), pool


def _cuts(T, n):
    """n packed prompts of T tokens in all, from short ones to long ones."""
    w = [i + 1 for i in range(n)]
    at = [0]
    for i in range(n):
        at.append(max(at[-1], T * sum(w[:i + 1]) // sum(w)))
    return at


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * (seed + 1) + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if c["op"] == "attn":
        order = torch.randperm(c["N"], generator=gen, device=DEV).tolist()
        full = _lengths(c)
        lengths = [full[i] for i in order]
        table, pool = _pages(lengths, c["page"], gen)
        kv = (pool, c["page"], c["Hkv"], c["d"])
        # some key channels are larger than others, as after a trained projection
        chan = torch.exp(0.4 * normal(c["Hkv"], c["d"]))
        act = torch.float32 if c["cache"] == "f32" else torch.bfloat16
        s = dict(c, q=normal(c["N"], c["m"], c["Hq"], c["d"]).to(act),
                 k_cache=(normal(*kv) * chan).to(DTYPES[c["cache"]]),
                 v_cache=normal(*kv).to(DTYPES[c["cache"]]), table=table,
                 lens=torch.tensor(lengths, dtype=torch.int32, device=DEV), max_len=c["hi"],
                 scale=c["d"] ** -0.5, k_scale=None, v_scale=None)
        if c["cache"] == "e4m3":
            s["k_scale"] = torch.exp(0.3 * normal(c["Hkv"]))
            s["v_scale"] = torch.exp(0.3 * normal(c["Hkv"]))
        return s
    if c["op"] == "append":
        n = c["packed"] or c["B"]
        act = DTYPES[c["act"]]
        if c["packed"]:
            at = _cuts(c["T"], n)
            new = [at[i + 1] - at[i] for i in range(n)]
        else:
            at, new = None, [c["T"]] * n
        start = torch.randint(c["lo"], c["hi"] + 1, (n,), generator=gen, device=DEV,
                              dtype=torch.int32)
        # a table that reaches the last position; only the pages written now are of a real pool
        first = start.cpu()
        width = max(int(a) + b for a, b in zip(first, new)) // c["page"] + 1
        cols = torch.arange(width, device=DEV)[None, :]
        ends = start + torch.tensor(new, dtype=torch.int32, device=DEV)
        mine = (cols >= (start // c["page"])[:, None]) & (cols * c["page"] < ends[:, None])
        pool = sum(-(-x // c["page"]) + 1 for x in new)  # a run of x tokens may begin inside a page
        table = torch.full((n, width), -1, dtype=torch.int64, device=DEV)
        table[mine] = torch.randperm(pool, generator=gen, device=DEV)[:int(mine.sum())]
        kv = (pool, c["page"], c["Hkv"], c["d"])
        tok = (c["B"], c["T"])
        s = dict(c, q=normal(*tok, c["Hq"], c["d"]).to(act), k=normal(*tok, c["Hkv"], c["d"]).to(act),
                 v=normal(*tok, c["Hkv"], c["d"]).to(act),
                 k_cache=torch.zeros(kv, device=DEV).to(DTYPES[c["cache"]]),
                 v_cache=torch.zeros(kv, device=DEV).to(DTYPES[c["cache"]]),
                 table=table.to(torch.int32), start=start, inv_freq=None, k_scale=None, v_scale=None,
                 cu=None if at is None else torch.tensor(at, dtype=torch.int32, device=DEV))
        if c["rot"]:
            i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
            s["inv_freq"] = (1e6 ** (-2.0 * i / c["rot"])).float()
        if c["cache"] == "e4m3":
            s["k_scale"] = torch.exp(0.3 * normal(c["Hkv"]))
            s["v_scale"] = torch.exp(0.3 * normal(c["Hkv"]))
        return s
    N, m, V = c["N"], c["m"], c["V"]
    logits = 3.0 * normal(N, m + 1, V)
    p = torch.softmax(logits, -1)
    draft = logits[:, :m] + 0.6 * normal(N, m, V)
    del logits
    q = torch.softmax(draft, -1).to(DTYPES[c["probs"]]) if c["drawn"] else None
    if c["drawn"]:  # a draw from q: the largest of the logits with Gumbel noise
        draft -= torch.log(-torch.log(torch.rand(N, m, V, generator=gen, device=DEV)
                                      .clamp_(1e-30, 1 - 1e-7)))
    x = draft.argmax(-1).to(torch.int32)
    del draft
    s = dict(c, p=p.to(DTYPES[c["probs"]]), q=q, x=x,
             r=torch.rand(N, m + 1, generator=gen, device=DEV), count=None)
    if c["ragged"]:
        s["count"] = torch.randint(0, m + 1, (N,), generator=gen, device=DEV, dtype=torch.int32)
    return s


# ------------------------------------------------------------------- the operators themselves

def run(s):
    if own:
        from gated_delta_rule_59_amd import binding
        if s["op"] == "attn":
            return binding.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                        scale=s["scale"], window=s["window"], max_len=s["max_len"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"],
                                        out_dtype=s["q"].dtype)
        if s["op"] == "append":
            q = binding.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["start"],
                                  q=s["q"], inv_freq=s["inv_freq"], interleaved=s["interleaved"],
                                  cu_seqlens=s["cu"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return q, s["k_cache"], s["v_cache"]
        return binding.verify_drafts(s["p"], s["q"], s["x"], s["r"], n_drafts=s["count"])
    return {"attn": _attn, "append": _append, "verify": _verify}[s["op"]](s)


def _attn(s):
    q, table, lens = s["q"], s["table"].long().clamp_min(0), s["lens"].long()
    N, m, Hq, d = q.shape
    Hkv, page = s["Hkv"], s["page"]
    L = table.shape[1] * page
    hi = lens[:, None] - m + 1 + torch.arange(m, device=DEV)                      # [N, m]
    lo = (hi - s["window"]).clamp_min(0) if s["window"] else torch.zeros_like(hi)
    t = torch.arange(L, device=DEV)
    seen = (t >= lo[..., None]) & (t < hi[..., None])                             # [N, m, L]
    k = s["k_cache"][table].float().view(N, L, Hkv, d).permute(0, 2, 3, 1)        # [N, Hkv, d, L]
    qf = q.float().view(N, m, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(N, Hkv, -1, d)
    x = torch.matmul(qf, k) * s["scale"]
    if s["k_scale"] is not None:
        x = x * s["k_scale"][:, None, None]
    mask = seen[:, None, :, None, :].expand(N, Hkv, m, Hq // Hkv, L).reshape(x.shape)
    x = x.masked_fill(~mask, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total > 0, total, torch.ones_like(total))
    v = s["v_cache"][table].float().view(N, L, Hkv, d).permute(0, 2, 1, 3)
    o = torch.matmul(x, v)
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None]
    return o.view(N, Hkv, m, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(N, m, Hq, d).to(q.dtype)


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, d] in 32 bits; cos, sin [tokens, 1, rot / 2]."""
    half = cos.shape[-1]
    if not half:
        return x
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _append(s):
    B, T, Hkv, d = s["k"].shape
    t = torch.arange(B * T, device=DEV)
    if s["cu"] is None:
        n, j = t // T, t % T
    else:
        cu = s["cu"].long()
        n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        j = t - cu[n]
    pos = s["start"].long()[n] + j
    slot = s["table"].long()[n, pos // s["page"]] * s["page"] + pos % s["page"]
    f = s["inv_freq"] if s["inv_freq"] is not None else torch.zeros(0, device=DEV)
    angle = pos.double()[:, None, None] * f.double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(s["q"].float().view(B * T, -1, d), cos, sin, s["interleaved"])
    k = _rotate(s["k"].float().view(B * T, Hkv, d), cos, sin, s["interleaved"])
    v = s["v"].float().view(B * T, Hkv, d)
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
    kind = torch.uint8 if s["cache"] == "e4m3" else s["k_cache"].dtype
    s["k_cache"].view(kind).view(-1, Hkv, d)[slot] = k.to(s["k_cache"].dtype).view(kind)
    s["v_cache"].view(kind).view(-1, Hkv, d)[slot] = v.to(s["v_cache"].dtype).view(kind)
    return q.to(s["q"].dtype).view(s["q"].shape), s["k_cache"], s["v_cache"]


def _verify(s):
    p, q, x, r = s["p"], s["q"], s["x"].long(), s["r"].double()
    N, m = x.shape
    rows = torch.arange(N, device=DEV)
    count = s["count"].long() if s["count"] is not None else torch.full((N,), m, device=DEV)
    px = p[:, :m].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    stands = (r[:, :m] * qx < px) & (torch.arange(m, device=DEV) < count[:, None])
    a = stands.long().cumprod(1).sum(1)
    last = a.clamp_max(m - 1)
    pa = p[rows, a].double()
    if q is not None:
        qa = q[rows, last].double()
    else:
        qa = torch.zeros_like(pa).scatter_(1, x[rows, last][:, None], 1.0)
    w = torch.where((a < count)[:, None], (pa - qa).clamp_min(0), pa)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, pa)
    c = w.cumsum(1)
    following = (c <= (r[:, m] * c[:, -1])[:, None]).sum(1)
    j = torch.arange(m + 1, device=DEV)[None, :]
    kept = torch.cat((x, x[:, :1]), 1)
    tokens = torch.where(j < a[:, None], kept, torch.where(j == a[:, None], following[:, None], -1))
    return a.to(torch.int32), tokens.to(torch.int32)


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "attn":
        lens = _lengths(c)
        seen = [min(x, c["window"] + c["m"] - 1) if c["window"] else x for x in lens]
        row = c["Hkv"] * c["d"] * BYTES[c["cache"]]
        act = 4 if c["cache"] == "f32" else 2
        qo = 2 * c["N"] * c["m"] * c["Hq"] * c["d"] * act
        return {"bytes": 2 * sum(seen) * row + qo, "flops": 4 * sum(seen) * c["m"] * c["Hq"] * c["d"]}
    if c["op"] == "append":
        tokens = c["B"] * c["T"] * c["d"]
        act = BYTES[c["act"]]
        return {"bytes": tokens * (2 * c["Hq"] * act + 2 * c["Hkv"] * (act + BYTES[c["cache"]])),
                "flops": 3 * c["B"] * c["T"] * c["rot"] * (c["Hq"] + c["Hkv"])}
    # the row of p that decides, and that of q where a draft fell (about seven drafts in ten stand)
    rows = 2.0 - 0.7 ** c["m"] if c["drawn"] else 1.0
    return {"bytes": c["N"] * c["V"] * BYTES[c["probs"]] * rows, "flops": 3 * c["N"] * c["V"]}


# --------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _attn64, "append": _append64, "verify": _verify64}[s["op"]](s)


def _attn64(s):
    """One sequence at a time, straight from the definition."""
    N, m, Hq, d = s["q"].shape
    group = Hq // s["Hkv"]
    out = torch.zeros(N, m, Hq, d, dtype=torch.float64, device=DEV)
    ks = s["k_scale"].double() if s["k_scale"] is not None else torch.ones(s["Hkv"], device=DEV).double()
    vs = s["v_scale"].double() if s["v_scale"] is not None else torch.ones(s["Hkv"], device=DEV).double()
    for n, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        ids = s["table"][n, :-(-length // s["page"])].long()
        keys = s["k_cache"][ids].flatten(0, 1)[:length].double() * ks[:, None]
        vals = s["v_cache"][ids].flatten(0, 1)[:length].double() * vs[:, None]
        for j in range(m):
            end = length - m + 1 + j
            begin = max(0, end - s["window"]) if s["window"] else 0
            if end <= 0:
                continue
            q = s["q"][n, j].double().view(s["Hkv"], group, d)
            z = torch.bmm(q, keys[begin:end].permute(1, 2, 0).contiguous()) * s["scale"]
            out[n, j] = torch.bmm(torch.softmax(z, -1),
                                  vals[begin:end].transpose(0, 1).contiguous()).view(Hq, d)
    return out


def _append64(s):
    """Every token as a complex rotation of its channel pairs."""
    B, T, Hkv, d = s["k"].shape
    at = s["cu"].tolist() if s["cu"] is not None else [i * T for i in range(B + 1)]
    first, half = s["start"].tolist(), s["rot"] // 2

    def turned(x, w):
        x = x.double()
        if not half:
            return x
        y = x.clone()
        i = torch.arange(half, device=DEV)
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(x[..., a], x[..., b]) * w
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q_out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV).view(B * T, -1, d)
    kc = s["k_cache"].double()
    vc = s["v_cache"].double()
    q, k, v = (s[x].reshape(B * T, -1, d) for x in ("q", "k", "v"))
    for n in range(len(at) - 1):
        a, b = at[n], at[n + 1]
        if a == b:
            continue
        pos = first[n] + torch.arange(b - a, device=DEV)
        w = None
        if half:
            theta = pos.double()[:, None, None] * s["inv_freq"].double()
            w = torch.polar(torch.ones_like(theta), theta)
        q_out[a:b] = turned(q[a:b], w)
        kn, vn = turned(k[a:b], w), v[a:b].double()
        if s["k_scale"] is not None:
            kn = (kn / s["k_scale"].double()[:, None]).clamp(-448, 448)
            vn = (vn / s["v_scale"].double()[:, None]).clamp(-448, 448)
        page = s["table"][n].long()[pos // s["page"]]
        kc[page, pos % s["page"]] = kn
        vc[page, pos % s["page"]] = vn
    return q_out.view(s["q"].shape), kc, vc


def _verify64(s):
    """One sequence after the other, one draft after the other."""
    N, m = s["x"].shape
    accept, tokens = [], []
    counts = s["count"].tolist() if s["count"] is not None else [m] * N
    for n in range(N):
        x, r = s["x"][n].tolist(), s["r"][n].double().tolist()
        a = 0
        while a < counts[n]:
            stand = float(s["q"][n, a, x[a]]) if s["q"] is not None else 1.0
            if not r[a] * stand < float(s["p"][n, a, x[a]]):
                break
            a += 1
        w = s["p"][n, a].double()
        if a < counts[n]:
            less = w.clone()
            if s["q"] is not None:
                less -= s["q"][n, a].double()
            else:
                less[x[a]] = 0.0
            less = less.clamp_min(0)
            w = less if float(less.sum()) > 0 else w
        c = torch.cumsum(w, 0)
        past = torch.nonzero(c > r[m] * c[-1])
        accept.append(a)
        tokens.append(x[:a] + [int(past[0])] + [-1] * (m - a))
    return (torch.tensor(accept, dtype=torch.int32, device=DEV),
            torch.tensor(tokens, dtype=torch.int32, device=DEV))
