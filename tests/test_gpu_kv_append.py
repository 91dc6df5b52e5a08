"""kda_kv_append against the 64-bit definition: rotation forms and far positions, cache types,
dense and packed batches, strides, slots that must stay as they are."""
import numpy as np
import pytest

from tests.paged_ref import STEP, U32, rotate

pytestmark = pytest.mark.gpu

FILL = 7.0


def freqs(rot, base=1e4):
    return (base ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32) if rot else None


def make(seed, starts, new, Hq, Hkv, d, rot, page, act, cache, packed=False, tail=0):
    """starts, new: cached and new tokens per sequence; tail: tokens behind the last one."""
    import torch
    rng = np.random.default_rng(seed)
    at = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    ct = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[cache]
    n = len(starts)
    B, T = (1, sum(new) + tail) if packed else (n, new[0])
    draw = lambda h: torch.from_numpy(  # noqa: E731
        rng.standard_normal((B, T, h, d)).astype(np.float32)).to(at).cuda()
    width = max(1, max((s + x - 1) // page + 1 for s, x in zip(starts, new)))
    table = np.full((n, width), -1)
    pool = 2
    for i in range(n):
        for pg in range(starts[i] // page, (starts[i] + new[i] - 1) // page + 1 if new[i] else 0):
            table[i, pg] = pool
            pool += 1
    perm = rng.permutation(pool)
    table = np.where(table >= 0, perm[np.maximum(table, 0)], -1)
    f = freqs(rot)
    dev = dict(k=draw(Hkv), v=draw(Hkv), q=draw(Hq),
               k_cache=torch.full((pool, page, Hkv, d), FILL, device="cuda").to(ct),
               v_cache=torch.full((pool, page, Hkv, d), FILL, device="cuda").to(ct),
               block_table=torch.from_numpy(table.astype(np.int32)).cuda(),
               start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
               inv_freq=None if f is None else torch.from_numpy(f).cuda())
    scale = np.ones((2, Hkv), np.float32)
    if cache == "e4m3":
        scale = np.exp(rng.standard_normal((2, Hkv)) * 0.3).astype(np.float32)
        dev["k_scale"], dev["v_scale"] = (torch.from_numpy(x.copy()).cuda() for x in scale)
    if packed:
        dev["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32,
                                         device="cuda")
    return dev, dict(starts=starts, new=new, table=table, f=f, scale=scale, page=page, act=act,
                     cache=cache, packed=packed, B=B, T=T)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def turn_bound(x, rot):
    """Sine and cosine are off by at most 4 units of 2^-24, the two products and their sum round
    three times: 8 units of 2^-24 of the pair's size (at most the row's largest twice)."""
    return 8 * U32 * 2 * np.abs(x).max() if rot else 0.0


def check(dev, h, q_out, pairs, skip=()):
    """Every cache slot and every row of q_out. skip: (sequence, j) that are not stored."""
    q, k, v = (host(dev[x]).reshape(h["B"] * h["T"], -1, dev[x].shape[-1]) for x in ("q", "k", "v"))
    qo = host(q_out).reshape(q.shape)
    kc, vc = host(dev["k_cache"]), host(dev["v_cache"])
    touched = np.zeros(kc.shape[:2], bool)
    f = h["f"] if h["f"] is not None else np.zeros(0, np.float32)
    cs, os_ = STEP[h["cache"]], STEP[h["act"]]
    # below 2^-6 an e4m3 step is 2^-9 whatever the value: half of it is 2^-10
    flat = 2.0 ** -10 if h["cache"] == "e4m3" else 0.0
    tok = 0
    for n, x in enumerate(h["new"]):
        for j in range(x):
            pos = h["starts"][n] + j
            t = tok + j
            ref = rotate(q[t], pos, f, pairs)
            assert (np.abs(qo[t] - ref) <= turn_bound(q[t], len(f)) + os_ * np.abs(ref)).all()
            if (n, j) in skip:
                continue
            pg, slot = h["table"][n, pos // h["page"]], pos % h["page"]
            touched[pg, slot] = True
            for c, val, s in ((kc, rotate(k[t], pos, f, pairs), h["scale"][0]), (vc, v[t], h["scale"][1])):
                ref = val / s[:, None]
                if h["cache"] == "e4m3":
                    ref = np.clip(ref, -448, 448)
                b = (turn_bound(k[t], len(f)) / s.min() if c is kc else 0.0) + 3 * U32 * np.abs(ref)
                b = b + cs * (np.abs(ref) + b) + flat
                assert (np.abs(c[pg, slot] - ref) <= b).all(), (n, j)
        tok += x
    fill = FILL
    assert (kc[~touched] == fill).all() and (vc[~touched] == fill).all()


CASES = [
    # starts, new, Hq, Hkv, d, rot, page, act, cache, packed, pairs
    ([0, 15, 16, 1000003], [1] * 4, 8, 2, 128, 128, 16, "bf16", "bf16", False, False),
    ([0, 5, 100], [3] * 3, 6, 3, 64, 32, 4, "bf16", "bf16", False, True),
    ([0, 5, 100], [3] * 3, 4, 4, 32, 16, 1, "bf16", "bf16", False, False),
    ([7, 0, 131071], [4] * 3, 5, 1, 64, 64, 48, "f32", "f32", False, False),
    ([7, 0, 131071], [4] * 3, 5, 1, 128, 96, 20, "f32", "f32", False, True),
    ([9, 31], [5] * 2, 2, 2, 128, 0, 16, "bf16", "bf16", False, False),
    ([3, 0, 40, 77, 0], [17, 0, 1, 30, 2], 4, 2, 128, 128, 16, "bf16", "bf16", True, False),
    ([3, 0, 40, 77, 0], [17, 0, 1, 30, 2], 4, 2, 64, 48, 7, "bf16", "e4m3", True, True),
    ([0, 65535], [6] * 2, 8, 8, 128, 128, 32, "bf16", "e4m3", False, False),
    ([0, 65535], [6] * 2, 3, 1, 32, 32, 32, "bf16", "e4m3", False, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_definition(case):
    import torch
    from gated_delta_rule_59_amd import binding
    starts, new, Hq, Hkv, d, rot, page, act, cache, packed, pairs = CASES[case]
    print(f"kv append {CASES[case]}", flush=True)
    dev, h = make((51, case), starts, new, Hq, Hkv, d, rot, page, act, cache, packed)
    q_out = binding.kv_append(**dev, interleaved=pairs)
    torch.cuda.synchronize()
    check(dev, h, q_out, pairs)


def test_many_packed_sequences_and_a_tail():
    """More sequences than a workgroup has threads; tokens behind the last one change nothing, in
    q_out neither."""
    import torch
    from gated_delta_rule_59_amd import binding
    rng = np.random.default_rng([52, 1])
    new = [int(x) for x in rng.integers(0, 3, 700)]
    starts = [int(x) for x in rng.integers(0, 50, 700)]
    dev, h = make((52, 2), starts, new, 2, 1, 32, 32, 16, "bf16", "bf16", packed=True, tail=5)
    q_out = torch.full_like(dev["q"], FILL)
    assert binding.kv_append(**dev, q_out=q_out) is q_out
    torch.cuda.synchronize()
    check(dev, h, q_out, False)
    assert (q_out[0, sum(new):] == FILL).all()


def test_without_queries_in_place_and_views():
    import torch
    from gated_delta_rule_59_amd import binding
    dev, h = make((53, 1), [4, 90], [3, 3], 4, 2, 64, 64, 16, "bf16", "bf16")
    fresh = lambda: {x: dev[x].clone() if x.endswith("_cache") else dev[x] for x in dev}  # noqa: E731
    a = fresh()
    qa = binding.kv_append(**a)
    b = fresh()
    del b["q"]
    assert binding.kv_append(**b) is None
    c = fresh()
    c["q"] = dev["q"].clone()
    qc = binding.kv_append(**c, q_out=c["q"])                       # q turned in place
    e = fresh()
    fused = torch.cat((dev["q"], dev["k"], dev["v"]), 2)              # views of one projection
    e["q"], e["k"], e["v"] = fused[:, :, :4], fused[:, :, 4:6], fused[:, :, 6:]
    qe = binding.kv_append(**e)
    # both caches in one allocation, heads outermost
    g = fresh()
    pool, page, H, d = dev["k_cache"].shape
    both = torch.full((pool, 2, H, page, d), FILL, device="cuda").to(torch.bfloat16)
    g["k_cache"], g["v_cache"] = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    qg = binding.kv_append(**g)
    torch.cuda.synchronize()
    check(a, h, qa, False)
    for x, q in ((b, qa), (c, qc), (e, qe), (g, qg)):
        assert torch.equal(q, qa)
        assert torch.equal(x["k_cache"], a["k_cache"]) and torch.equal(x["v_cache"], a["v_cache"])


def test_positions_and_pages_out_of_range():
    """Tokens past the table, before position 0 or on no page are not stored; all else is."""
    import torch
    from gated_delta_rule_59_amd import binding
    starts, page = [14, 14, 14, 14], 16
    dev, h = make((54, 1), starts, [4] * 4, 2, 1, 32, 0, page, "bf16", "bf16")
    width = dev["block_table"].shape[1]
    assert width == 2
    dev["block_table"][0, 1] = dev["k_cache"].shape[0]
    dev["block_table"][1, 0] = -1
    dev["start"][2] = 2 * page - 1
    dev["start"][3] = -2
    h["starts"] = [14, 14, 2 * page - 1, -2]
    skip = {(0, 2), (0, 3), (1, 0), (1, 1), (2, 1), (2, 2), (2, 3), (3, 0), (3, 1)}
    q_out = binding.kv_append(**dev)
    torch.cuda.synchronize()
    check(dev, h, q_out, False, skip)


def test_e4m3_limits_and_nan():
    import torch
    from gated_delta_rule_59_amd import binding
    dev, h = make((55, 1), [0], [1], 1, 1, 32, 0, 16, "bf16", "e4m3")
    dev["k_scale"].fill_(0.5)
    x = torch.zeros(32)
    x[:10] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 224.0, 1.0625, 1.1875, 2.0 ** -10, 0.0])
    dev["k"][0, 0, 0] = x.to(torch.bfloat16).cuda()
    binding.kv_append(**dev)
    torch.cuda.synchronize()
    pg = int(dev["block_table"][0, 0])
    got = dev["k_cache"][pg, 0, 0].float().cpu()
    want = (dev["k"][0, 0, 0].float() / 0.5).clamp(-448, 448).cpu().to(torch.float8_e4m3fn).float()
    assert torch.isnan(got[4])
    want[4] = got[4] = 0
    assert torch.equal(got, want)


def test_e4m3_quotients_that_are_ties():
    """Odd multiples of 7 over a scale of 7 lie halfway between two e4m3 values and go to the even
    one; times the rounded 1 / 7 they come out above the middle."""
    import torch
    from gated_delta_rule_59_amd import binding
    dev, h = make((55, 2), [0], [1], 1, 1, 32, 0, 16, "bf16", "e4m3")
    dev["k_scale"].fill_(7.0)
    dev["v_scale"].fill_(7.0)
    x = torch.zeros(32)
    x[:10] = torch.tensor([161.0, 175.0, 189.0, 203.0, 217.0, -161.0, -175.0, -189.0, -203.0, -217.0])
    for name in ("k", "v"):
        dev[name][0, 0, 0] = x.to(torch.bfloat16).cuda()
    binding.kv_append(**dev)
    torch.cuda.synchronize()
    pg = int(dev["block_table"][0, 0])
    want = torch.zeros(32)
    want[:10] = torch.tensor([24.0, 24.0, 28.0, 28.0, 32.0, -24.0, -24.0, -28.0, -28.0, -32.0])
    for c in ("k_cache", "v_cache"):
        assert torch.equal(dev[c][pg, 0, 0].float().cpu(), want)


def test_no_tokens():
    import torch
    from gated_delta_rule_59_amd import binding
    dev, h = make((56, 1), [3], [1], 1, 1, 32, 32, 16, "bf16", "bf16")
    for x in ("q", "k", "v"):
        dev[x] = dev[x][:, :0]
    assert binding.kv_append(**dev).shape == (1, 0, 1, 32)
    torch.cuda.synchronize()
    assert (dev["k_cache"] == FILL).all()


def test_captured_and_replayed_on_another_stream():
    import torch
    from gated_delta_rule_59_amd import binding
    dev, h = make((57, 1), [10, 30], [2, 2], 4, 2, 64, 64, 16, "bf16", "bf16")
    ref = {x: dev[x].clone() if x.endswith("_cache") else dev[x] for x in dev}
    want = binding.kv_append(**ref)
    torch.cuda.synchronize()
    check(ref, h, want, False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q_out = binding.kv_append(**dev)
    for _ in range(3):
        dev["k_cache"].fill_(FILL)
        dev["v_cache"].fill_(FILL)
        q_out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want)
        assert torch.equal(dev["k_cache"], ref["k_cache"]) and torch.equal(dev["v_cache"], ref["v_cache"])
    dev["k_cache"].fill_(FILL)
    dev["v_cache"].fill_(FILL)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q2 = binding.kv_append(**dev, stream=s)
    s.synchronize()
    assert torch.equal(q2, want) and torch.equal(dev["v_cache"], ref["v_cache"])


def test_binding_refuses_what_it_cannot_pass_on():
    import torch
    from gated_delta_rule_59_amd import binding
    dev, _ = make((58, 1), [4, 90], [3, 3], 4, 2, 64, 64, 16, "bf16", "bf16")
    call = lambda **kw: binding.kv_append(**{**dev, **kw})  # noqa: E731
    wide = torch.zeros((2, 5, 2, 64), dtype=torch.bfloat16, device="cuda")
    for error, match, kw in [
            (ValueError, "evenly", dict(k=wide[:, :3])), (TypeError, "q must be", dict(q=dev["q"].float())),
            (TypeError, "start", dict(start=dev["start"].long())), (ValueError, "start", dict(start=dev["start"][:1])),
            (ValueError, "must be on", dict(start=dev["start"].cpu())),
            (ValueError, "must be on", dict(k_cache=dev["k_cache"].cpu())),
            (TypeError, "k_cache", dict(k_cache=dev["k_cache"].half())),
            (ValueError, "k_cache", dict(k_cache=dev["k_cache"][:, :, :1])),
            (ValueError, "channels", dict(v_cache=dev["v_cache"].transpose(2, 3).contiguous().transpose(2, 3))),
            (TypeError, "block_table", dict(block_table=dev["block_table"].long())),
            (ValueError, "block_table", dict(block_table=dev["block_table"][:1])),
            (ValueError, "q_out", dict(q_out=torch.empty_like(wide))), (ValueError, "q_out needs q", dict(q=None, q_out=dev["q"])),
            (binding.KDAError, "F8E4M3", dict(k_scale=torch.ones(2, device="cuda"))),
            (binding.KDAError, "rot", dict(inv_freq=torch.ones(40, device="cuda"))),
            (binding.KDAError, "overlaps", dict(q_out=dev["k_cache"].view(-1)[:dev["q"].numel()].view(dev["q"].shape)))]:
        with pytest.raises(error, match=match):
            call(**kw)
    with pytest.raises(binding.KDAError) as e:
        call(inv_freq=torch.ones(20, device="cuda"))
    assert e.value.status == 2
    torch.cuda.synchronize()
    assert (dev["k_cache"] == FILL).all()
