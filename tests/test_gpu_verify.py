"""kda_verify_drafts against the 64-bit definition (whole numbers: equal), and the distribution it
leaves; then a whole speculative step of a hybrid stack with kda_decode_multi."""
import numpy as np
import pytest

from tests.paged_ref import verify

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(seed, N, m, V, drawn=True, spread=3.0):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((N, m + 1, V)) * spread
    p = softmax(logits)
    d = logits[:, :m] + 0.7 * rng.standard_normal((N, m, V))
    q = softmax(d) if drawn else None
    if drawn:
        x = (d + rng.gumbel(size=d.shape)).argmax(-1).astype(np.int32)
    else:
        x = d.argmax(-1).astype(np.int32)
    return p, q, x, rng.random((N, m + 1)).astype(np.float32)


def run(p, q, x, r, counts=None, dtype="f32", **kw):
    """Device result, and the host values the device saw."""
    import torch
    from gated_delta_rule_59_amd import binding
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    tp = torch.from_numpy(p).to(t).cuda()
    tq = None if q is None else torch.from_numpy(q).to(t).cuda()
    n = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    a, tok = binding.verify_drafts(tp, tq, torch.from_numpy(x).cuda(), torch.from_numpy(r).cuda(),
                                   n_drafts=n, **kw)
    torch.cuda.synchronize()
    return (a.cpu().numpy(), tok.cpu().numpy(), tp.float().cpu().numpy(),
            None if q is None else tq.float().cpu().numpy())


def check(p, q, x, r, counts=None, dtype="f32", **kw):
    a, tok, hp, hq = run(p, q, x, r, counts, dtype, **kw)
    ra, rt = verify(hp, hq, x, r, counts if counts is not None else [x.shape[1]] * len(x))
    assert (a == ra).all(), (a, ra)
    assert (tok == rt).all(), (tok, rt)
    return a


@pytest.mark.parametrize("N,m,V,drawn,dtype", [
    (1, 1, 1, True, "f32"), (3, 2, 7, True, "f32"), (40, 4, 1000, True, "f32"),
    (17, 4, 2048, True, "f32"), (17, 3, 2049, False, "f32"), (9, 8, 50257, True, "bf16"),
    (5, 1, 32000, False, "bf16"), (6, 5, 131073, True, "f32"), (2, 300, 33, True, "f32"),
    (2, 2, 600001, True, "f32")])
def test_against_definition(N, m, V, drawn, dtype):
    print(f"verify N={N} m={m} V={V} drawn={drawn} {dtype}", flush=True)
    p, q, x, r = make((61, N, m, V), N, m, V, drawn)
    a = check(p, q, x, r, dtype=dtype)
    if N >= 17 and drawn:
        assert a.min() == 0 and a.max() == m   # both ways of choosing the following token


@pytest.mark.parametrize("N,m,V,drawn,dtype", [
    (3, 2, 16384, True, "f32"), (3, 2, 16385, True, "f32"), (2, 3, 16383, True, "bf16"), (2, 3, 16400, False, "bf16"),
    (256, 2, 1025, True, "f32"), (257, 2, 1025, True, "f32"), (300, 1, 3, False, "f32")])
def test_one_launch_or_two(N, m, V, drawn, dtype):
    """Around the vocabulary and the number of sequences up to which one workgroup does a sequence."""
    print(f"verify N={N} m={m} V={V} drawn={drawn} {dtype}", flush=True)
    p, q, x, r = make((66, N, m, V), N, m, V, drawn)
    check(p, q, x, r, dtype=dtype)


def test_ragged_counts():
    p, q, x, r = make((62, 1), 24, 4, 500)
    check(p, q, x, r, counts=[0, 1, 2, 3, 4, -3, 9, 4] * 3)
    check(p, None, x, r, counts=[0, 1, 2, 3, 4, -3, 9, 4] * 3)


def test_the_same_distribution_always_stands():
    """q = p: every draft stands (uniform numbers are below 1)."""
    p, _, x, r = make((63, 1), 12, 3, 257)
    a = check(p, np.ascontiguousarray(p[:, :3]), x, r)
    assert (a[[i for i in range(12) if (p[i, range(3), x[i]] > 0).all()]] == 3).all()


def test_extreme_uniform_numbers():
    """0, the largest below 1, and values out of range, for drafts and for the following token."""
    p, q, x, r = make((64, 1), 8, 2, 3000, spread=6.0)
    top = np.nextafter(np.float32(1), np.float32(0))
    r[:, 2] = [0, top, 1, 2, -1, np.nan, np.inf, -np.inf]
    with np.errstate(invalid="ignore"):
        check(p, q, x, r)
        r[:, 0] = [0, top, 1, 2, -1, np.nan, np.inf, -np.inf]
        check(p, q, x, r)


def test_bad_probabilities_and_drafts():
    """NaN, infinities, negative values and rows of zeros; drafts that are no tokens."""
    p, q, x, r = make((65, 1), 10, 2, 700)
    p[0, 0] = 0
    p[1, :] = 0
    p[2, 0, 5:400:7] = np.nan
    p[3, 0, 3:600:5] = np.inf
    p[4, 0] = -p[4, 0]
    q[5, 0] = np.nan
    q[6, 0, x[6, 0]] = np.inf
    x[7, 0], x[8, 0], x[9, 1] = -1, 700, 2 ** 31 - 1
    q[1, 0] = p[1, 0]
    check(p, q, x, r)
    check(p, None, x, r)


def test_residual_of_nothing_falls_back_to_the_target():
    """A draft with p = 0 where q covers all of p: max(p - q, 0) is zero everywhere."""
    V = 64
    p = np.zeros((1, 2, V), np.float32)
    p[0, 0, :32] = 1 / 64
    p[0, 1] = 1 / V
    q = np.full((1, 1, V), 1 / 64, np.float32)
    for u in (0.0, 0.3, 0.99):
        check(p, q, np.array([[40]], np.int32), np.array([[0.5, u]], np.float32))


def test_strided_rows():
    """Rows of a padded vocabulary, the target's and the draft's with different strides."""
    import torch
    from gated_delta_rule_59_amd import binding
    p, q, x, r = make((66, 1), 5, 3, 1001)
    tp = torch.full((5, 6, 1024), float("nan"), device="cuda")
    tq = torch.full((5, 3, 1003), float("nan"), device="cuda")
    tp[:, 1:5, :1001] = torch.from_numpy(p)
    tq[:, :, 2:] = torch.from_numpy(q)
    a, tok = binding.verify_drafts(tp[:, 1:5, :1001], tq[:, :, 2:], torch.from_numpy(x).cuda(),
                                   torch.from_numpy(r).cuda())
    torch.cuda.synchronize()
    ra, rt = verify(p, q, x, r, [3] * 5)
    assert (a.cpu().numpy() == ra).all() and (tok.cpu().numpy() == rt).all()


def test_following_token_is_distributed_as_the_target():
    """One draft from q, verified 200,000 times: the first token's frequencies are p's (within five
    standard deviations each)."""
    N, V = 200000, 5
    rng = np.random.default_rng([67, 1])
    p1 = np.array([0.1, 0.2, 0.3, 0.4, 0.0], np.float32)
    q1 = np.array([0.4, 0.1, 0.1, 0.2, 0.2], np.float32)
    p = np.broadcast_to(p1, (N, 2, V)).copy()
    q = np.broadcast_to(q1, (N, 1, V)).copy()
    x = rng.choice(V, size=(N, 1), p=q1 / q1.sum(dtype=np.float64)).astype(np.int32)
    _, tok, _, _ = run(p, q, x, rng.random((N, 2)).astype(np.float32))
    f = np.bincount(tok[:, 0], minlength=V) / N
    sd = np.sqrt(p1 * (1 - p1) / N)
    assert (np.abs(f - p1) <= 5 * sd + 1e-12).all(), f


def test_captured_and_replayed():
    import torch
    from gated_delta_rule_59_amd import binding
    cases = [make((68, i), 6, 3, 4000) for i in range(3)]
    dev = [torch.from_numpy(z).cuda() for z in cases[0]]
    binding.verify_drafts(*dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, tok = binding.verify_drafts(*dev)
    for i in (0, 1, 2, 0):
        for d, z in zip(dev, cases[i]):
            d.copy_(torch.from_numpy(z))
        g.replay()
        torch.cuda.synchronize()
        ra, rt = verify(*cases[i], [3] * 6)
        assert (a.cpu().numpy() == ra).all() and (tok.cpu().numpy() == rt).all()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        b, tok2 = binding.verify_drafts(*dev, stream=s)
        s.synchronize()
        assert torch.equal(a, b) and torch.equal(tok, tok2)


def test_speculative_step_of_a_hybrid_stack():
    """A step as a server runs it: four drafts' keys and values appended to the attention layer's
    pages, attention over them, the KDA layer's outputs of the drafts, the verification, and the
    commit of what stands: afterwards both layers are where token-by-token decoding of the accepted
    drafts takes them."""
    import torch
    import oracle
    from gated_delta_rule_59_amd import binding, inputs
    from tests.gpu_util import TAU, assert_parity, dev, host
    from tests.paged_ref import attend, attend_bound, rotate
    N, m, H, Hq, Hkv, d, page, V = 6, 4, 2, 8, 2, 128, 16, 1000
    rng = np.random.default_rng([69, 1])
    past = [0, 1, 15, 16, 33, 200]
    cap = max(past) + m
    width = -(-cap // page)
    table = torch.from_numpy(rng.permutation(N * width).reshape(N, width).astype(np.int32)).cuda()
    kc = torch.full((N * width, page, Hkv, d), float("nan"), device="cuda").to(torch.bfloat16)
    vc = kc.clone()
    f = torch.from_numpy((1e4 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)).cuda()
    lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    # the prompts, packed
    total = sum(past)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(past)]).astype(np.int32)).cuda()
    pk, pv = bf(1, total, Hkv, d), bf(1, total, Hkv, d)
    binding.kv_append(pk, pv, kc, vc, table, torch.zeros_like(lens), inv_freq=f, cu_seqlens=cu)
    # the drafts, at the attention layer
    q, k, v = bf(N, m, Hq, d), bf(N, m, Hkv, d), bf(N, m, Hkv, d)
    q_rot = binding.kv_append(k, v, kc, vc, table, lens, q=q, inv_freq=f)
    o = binding.paged_decode(q_rot, kc, vc, table, lens + m, max_len=cap)
    # the drafts, at the KDA layer
    x = inputs.draw_activations((69, 2), N, m, H, d, d, "bf16")
    S0 = inputs.draw_state((69, 2), N, H, d, d)
    tx = [dev(a, "bf16") for a in x]
    S = torch.from_numpy(S0).cuda()
    o_kda = binding.decode_multi(*tx, S)
    # which of them stand
    p, pq, drafts, r = make((69, 3), N, m, V)
    accept, tokens = binding.verify_drafts(*[torch.from_numpy(z).cuda() for z in (p, pq, drafts, r)])
    binding.decode_multi(*tx, S, accept=accept, want_output=False)
    lens = lens + accept
    torch.cuda.synchronize()

    ra, rt = verify(p, pq, drafts, r, [m] * N)
    assert (accept.cpu().numpy() == ra).all() and (tokens.cpu().numpy() == rt).all()
    h64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    hk, hv, hq, fr = h64(k), h64(v), h64(q), f.cpu().numpy()
    ks, vs, at = [], [], 0
    for n, L in enumerate(past):
        t = np.arange(L + m)
        pages = table[n].cpu().numpy()[t // page]
        ks.append(h64(kc)[pages, t % page])
        vs.append(h64(vc)[pages, t % page])
        want = np.array([rotate(h64(pk[0, at + i]), i, fr, False) for i in range(L)]
                        + [rotate(hk[n, j], L + j, fr, False) for j in range(m)])
        # one bf16 rounding, and the rotation's own (tests/test_gpu_kv_append.py: under 2^-20 of 4.5)
        assert (np.abs(ks[n] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17).all()
        assert (vs[n] == np.concatenate([h64(pv[0, at:at + L]), hv[n]])).all()
        at += L
    full = [L + m for L in past]
    ref, _ = attend(h64(q_rot), ks, vs, [np.ones(L, bool) for L in full], full, d ** -0.5, 0)
    tol = attend_bound(h64(q_rot), ks, vs, full, d ** -0.5, "bf16", ref, "f32")
    assert (np.abs(h64(o) - ref) <= tol).all()
    want = np.array([[rotate(hq[n, j], past[n] + j, fr, False) for j in range(m)] for n in range(N)])
    assert (np.abs(h64(q_rot) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17).all()
    o_ref, _ = oracle.kda_reference(*x, S0)
    assert_parity(host(o_kda), o_ref, TAU["bf16"], "KDA outputs of the drafts")
    cat = lambda a: np.concatenate([a[n, :ra[n]] for n in range(N)])[None]  # noqa: E731
    cuk = np.concatenate([[0], np.cumsum(ra)]).astype(np.int32)
    _, s_ref = oracle.kda_reference(*[cat(a) for a in x], S0, cu_seqlens=cuk)
    assert_parity(host(S), s_ref, TAU["bf16"], "committed states")
