"""Linear attention with a decay for each head against the recurrence in 64 bits: prompts, single tokens,
drafts.

Errors are bounded relative to the same sums over absolute values (ao, A of step_ref.lin). In units of
2^-24 = u: a product of dk terms in 32 bits dk u, sums over the 64 tokens of a chunk twice 64 u, one
rounding per chunk of the state; decays e^x with |x| up to 88 (beyond, they are 0), x rounded twice:
176 u < 2^-16; states and weights in bf16 parts 2^-16 together, in the state's own sum 2^-22. Then the
result's own rounding: 2^-8 relative for bf16, u for fp32."""
import numpy as np
import pytest

from tests.step_ref import lin

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def rounded(x, dtype):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return t.bfloat16().float().numpy() if dtype == "bf16" else t.numpy()


def dev(x, dtype="f32"):
    import torch
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def make(seed, T, Hk, H, dk, dv, n_seq, act="bf16", gate="f32", fixed=False, decay=1.0, first=True):
    rng = np.random.default_rng(seed)
    q, k = (rounded(rng.standard_normal((T, Hk, dk)), act) for _ in range(2))
    v = rounded(rng.standard_normal((T, H, dv)), act)
    rate = decay * 2.0 ** -np.linspace(8, -2, H)
    g = -rate if fixed else -rate * np.log1p(np.exp(rng.standard_normal((T, H))))
    S0 = rng.standard_normal((n_seq, H, dk, dv)).astype(np.float32) if first else None
    return q, k, v, rounded(g, gate), S0


def bounds(ref, ao, A, dk, T, out):
    o, S = ref
    steps = dk + 128 + T / 64 + 16
    eo = HALF[out] * np.abs(o) + (2.0 ** -15 + steps * U) * ao + 1e-35
    es = U * np.abs(S) + (2.0 ** -16 + 2.0 ** -22 + steps * U) * A + 1e-35
    return eo, es


def close(got, want, bound, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{what}: {np.nanmax(err / bound):.3g} of the bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def prompt(x, lengths=None, B=1, scale=0.3, act="bf16", gate="f32", out="f32", **kw):
    """lin_chunk_fwd of packed sequences or a dense batch, checked; returns (o, S_T)."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = x
    T = q.shape[0]
    cu = None
    if lengths is not None:
        cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32, device="cuda")
    lens = lengths if lengths is not None else [T // B] * B
    view = lambda t: t.view(B, T // B, *t.shape[1:])  # noqa: E731
    gd = dev(g, gate)
    o, S = binding.lin_chunk_fwd(view(dev(q, act)), view(dev(k, act)), view(dev(v, act)),
                                 gd if g.ndim == 1 else view(gd), dev(S0), cu, scale=scale,
                                 out_dtype=torch.float32 if out == "f32" else torch.bfloat16, **kw)
    torch.cuda.synchronize()
    ro, rS, ao, A = lin(q, k, v, g, S0, scale, lens)
    eo, es = bounds((ro, rS), ao, A, q.shape[2], max(lens), out)
    close(o, ro, eo, "o")
    close(S, rS, es, "S_T")
    return o, S


DIMS = [(a, b) for a in (32, 64, 128) for b in (32, 64, 128)]


@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_prompt_dims_and_types(dk, dv, act, out):
    print(f"lin prompt {dk}x{dv} {act}->{out}", flush=True)
    x = make((1, dk, dv), 2 * 203, 2, 4, dk, dv, 2, act)
    prompt(x, B=2, act=act, out=out)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prompt_lengths(T, act):
    print(f"lin prompt T={T} {act}", flush=True)
    prompt(make((2, T), T, 1, 3, 64, 128, 1, act, first=T % 2 == 0), act=act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prompt_of_many_segments(act):
    """One sequence and two heads: the longest chain of segments; long and short memory."""
    prompt(make((3, 1), 5000, 1, 2, 128, 128, 1, act, decay=0.02), act=act)


@pytest.mark.parametrize("lengths", [[0], [0, 5, 0], [64, 64, 1], [1] * 70, [700, 3, 0, 0, 129, 64, 31, 1200], [2, 1500]])
@pytest.mark.parametrize("first", [True, False])
def test_packed(lengths, first):
    print(f"lin packed {lengths}", flush=True)
    x = make((4, len(lengths)), sum(lengths), 2, 2, 64, 64, len(lengths), first=first)
    prompt(x, lengths)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("N,most,long", [(65, 200, 0), (200, 40, 3000), (1100, 9, 700), (64, 150, 2600)])
def test_many_packed(N, most, long, act):
    """More sequences than lanes of a wave or threads of a workgroup, empty ones and a long one among them."""
    print(f"lin packed {N} of up to {most} and {long} {act}", flush=True)
    lengths = [int(x) for x in np.random.default_rng((12, N)).integers(0, most + 1, N)]
    lengths[N // 2] = max(lengths[N // 2], long)
    prompt(make((13, N), sum(lengths), 1, 2, 32, 32, N, act), lengths, act=act)


@pytest.mark.parametrize("fixed,gate", [(True, "f32"), (True, "bf16"), (False, "bf16")])
def test_decay_forms(fixed, gate):
    prompt(make((5, fixed), 500, 3, 6, 32, 64, 1, gate=gate, fixed=fixed), gate=gate)


def test_decays_from_none_to_whole():
    """g = 0 (no decay), strong decays whose running sum dwarfs those after it, and -infinity, which ends
    the memory; growth too."""
    x = make((6, 1), 400, 2, 4, 64, 64, 1)
    g = x[3]
    g[:, 0] = 0
    g[::7, 1] = -60.0
    g[1::7, 1] = -1e-3
    g[40, 2] = g[64, 2] = g[65, 2] = g[399, 2] = -np.inf
    g[:, 3] = 0.01
    with np.errstate(invalid="ignore"):
        prompt(x)


def test_no_tokens():
    import torch
    from gated_delta_rule_59_amd import binding
    S0 = torch.randn(3, 2, 64, 32, device="cuda")
    z = torch.empty(3, 0, 2, 64, device="cuda")
    o, S = binding.lin_chunk_fwd(z, z, torch.empty(3, 0, 2, 32, device="cuda"), torch.empty(3, 0, 2, device="cuda"), S0)
    assert o.shape == (3, 0, 2, 32) and torch.equal(S, S0)
    _, S = binding.lin_chunk_fwd(z, z, torch.empty(3, 0, 2, 32, device="cuda"), torch.zeros(2, device="cuda"))
    assert torch.equal(S, torch.zeros_like(S0))
    S = S0.clone()
    binding.lin_chunk_fwd(z, z, torch.empty(3, 0, 2, 32, device="cuda"), torch.zeros(2, device="cuda"), S, S_T=S)
    assert torch.equal(S, S0)


def test_in_place_and_in_pieces():
    """S_T = S0, and a prompt in two calls; the states of both agree within the bound, in place bitwise."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((7, 1), 3000, 2, 4, 128, 64, 1)
    d = [dev(a, "bf16")[None] for a in (q, k, v)]
    gd = dev(g)[None]
    _, want = prompt((q, k, v, g, S0))
    S = dev(S0)
    o, out = binding.lin_chunk_fwd(*d, gd, S, S_T=S)
    assert out.data_ptr() == S.data_ptr() and torch.equal(S, want)
    S = dev(S0)
    for a, b in ((0, 1111), (1111, 3000)):
        binding.lin_chunk_fwd(*[t[:, a:b] for t in d], gd[:, a:b].contiguous(), S, S_T=S)
    ro, rS, ao, A = lin(q, k, v, g, S0, 1.0)
    close(S, rS, bounds((ro, rS), ao, A, 128, 3000, "f32")[1], "S in pieces")


def test_rows_behind_the_last_sequence_stay():
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((8, 1), 500, 2, 2, 64, 64, 2)
    cu = torch.tensor([0, 130, 333], dtype=torch.int32, device="cuda")
    o = torch.full((1, 500, 2, 64), 7.0, device="cuda")
    got, S = binding.lin_chunk_fwd(*[dev(a, "bf16")[None] for a in (q, k, v)], dev(g)[None], dev(S0), cu, o=o)
    assert got is o and (o[0, 333:] == 7.0).all()
    ro, rS, ao, A = lin(q[:333], k[:333], v[:333], g[:333], S0, 1.0, [130, 203])
    eo, es = bounds((ro, rS), ao, A, 64, 203, "f32")
    close(o[0, :333], ro, eo, "o")
    close(S, rS, es, "S")


def test_offsets_out_of_range_stay_in_bounds():
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((9, 1), 256, 1, 2, 64, 64, 4)
    cu = torch.tensor([-50, 100, 60, 256, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    _, S = binding.lin_chunk_fwd(*[dev(a, "bf16")[None] for a in (q, k, v)], dev(g)[None], dev(S0), cu)
    ro, rS, ao, A = lin(q[:100], k[:100], v[:100], g[:100], S0[:1], 1.0)
    close(S[:1], rS, bounds((ro, rS), ao, A, 64, 100, "f32")[1], "first")
    assert torch.equal(S[[1, 3]].cpu(), torch.from_numpy(S0[[1, 3]]))
    ro, rS, ao, A = lin(q[60:], k[60:], v[60:], g[60:], S0[2:3], 1.0)
    close(S[2:3], rS, bounds((ro, rS), ao, A, 64, 196, "f32")[1], "third")


def test_strided_views_of_one_projection():
    import torch
    from gated_delta_rule_59_amd import binding
    B, T, Hk, H, dk, dv = 2, 150, 2, 4, 64, 32
    q, k, v, g, S0 = make((10, 1), B * T, Hk, H, dk, dv, B)
    fused = torch.full((B, T, 2 * Hk * dk + H * dv + 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    qv = fused[..., 8:8 + Hk * dk].view(B, T, Hk, dk)
    kv = fused[..., 8 + Hk * dk:8 + 2 * Hk * dk].view(B, T, Hk, dk)
    vv = fused[..., 8 + 2 * Hk * dk:8 + 2 * Hk * dk + H * dv].view(B, T, H, dv)
    qv.copy_(dev(q, "bf16").view(B, T, Hk, dk)), kv.copy_(dev(k, "bf16").view(B, T, Hk, dk))
    vv.copy_(dev(v, "bf16").view(B, T, H, dv))
    gd = dev(g).view(B, T, H)
    got = binding.lin_chunk_fwd(qv, kv, vv, gd, dev(S0))
    want = prompt((q, k, v, g, S0), B=B, scale=1.0)
    assert all(torch.equal(a, b.view(a.shape)) for a, b in zip(got, want))
    # heads outermost, and one value head for all (stride 0)
    turned = [t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (qv, kv, vv)]
    if B == 1:
        got = binding.lin_chunk_fwd(*turned, gd, dev(S0))
        assert all(torch.equal(a, b.view(a.shape)) for a, b in zip(got, want))
    one = vv[:, :, :1].expand(B, T, H, dv)
    got = binding.lin_chunk_fwd(qv, kv, one, gd, dev(S0))
    want = binding.lin_chunk_fwd(qv.contiguous(), kv.contiguous(), one.contiguous(), gd, dev(S0))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_values_that_are_not_finite():
    """They stay in their sequence, in the heads that read them, and reach no token 64 or more before."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((11, 1), 400, 2, 4, 64, 64, 2)
    cu = torch.tensor([0, 190, 400], dtype=torch.int32, device="cuda")
    run = lambda v, k: binding.lin_chunk_fwd(dev(q, "bf16")[None], dev(k, "bf16")[None], dev(v, "bf16")[None],  # noqa: E731
                                             dev(g)[None], dev(S0), cu)
    want, Sw = run(v, k)
    v2, k2 = v.copy(), k.copy()
    v2[300, 1, 5] = np.nan
    k2[310, 1, 7] = np.inf    # key head 1: heads 2 and 3
    got, Sg = run(v2, k2)
    same = torch.ones(400, 4, dtype=torch.bool)
    same[300 - 63:, 1] = False
    same[310 - 63:, 2:] = False
    assert torch.equal(got[0].cpu()[same], want[0].cpu()[same])
    assert torch.equal(Sg[0], Sw[0]) and torch.equal(Sg[1, 0], Sw[1, 0])
    assert not torch.isfinite(got[0, 300:, 1, 5]).any() and not torch.isfinite(Sg[1, 1, :, 5]).any()


# ------------------------------------------------------------------------------ tokens and drafts

def token_bounds(ref, ao, A, dk, m, out):
    """All in 32 bits: the sums over dk and m, one rounding per token of the state, and the decay's."""
    o, S = ref
    steps = dk + 3 * m + 8 + 176
    return HALF[out] * np.abs(o) + steps * U * ao + 1e-35, U * np.abs(S) + (3 * m + 4 + 176) * U * A + 1e-35


@pytest.mark.parametrize("act,gate,out", [("bf16", "f32", "bf16"), ("f32", "bf16", "f32"), ("bf16", "bf16", "f32")])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_step(dk, dv, act, gate, out):
    import torch
    from gated_delta_rule_59_amd import binding
    print(f"lin step {dk}x{dv} {act} {gate} {out}", flush=True)
    N, Hk, H = 5, 2, 6
    q, k, v, g, S0 = make((20, dk, dv), N, Hk, H, dk, dv, N, act, gate)
    S = dev(S0)
    o = binding.lin_decode_step(dev(q, act), dev(k, act), dev(v, act), dev(g, gate), S, scale=0.4,
                                out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    ro, rS, ao, A = lin(q, k, v, g, S0, 0.4, [1] * N)
    eo, es = token_bounds((ro, rS), ao, A, dk, 1, out)
    assert o.shape == (N, H, dv)
    close(o, ro, eo, "o")
    close(S, rS, es, "S")


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 17])
@pytest.mark.parametrize("fixed", [False, True])
def test_drafts(m, fixed):
    """Verification leaves S, commits take any number of drafts, results agree bitwise."""
    import torch
    from gated_delta_rule_59_amd import binding
    N, Hk, H, dk, dv = 6, 1, 3, 128, 64
    q, k, v, g, S0 = make((21, m), N * m, Hk, H, dk, dv, N, fixed=fixed)
    view = lambda t: t.view(N, m, *t.shape[1:])  # noqa: E731
    d = [view(dev(a, "bf16")) for a in (q, k, v)]
    gd = dev(g) if fixed else view(dev(g))
    S = dev(S0)
    o = binding.lin_decode_multi(*d, gd, S, scale=0.4)
    assert torch.equal(S, dev(S0))
    ro, _, ao, A = lin(q, k, v, g, S0, 0.4, [m] * N)
    close(o, ro, token_bounds((ro, S0), ao, A, dk, m, "f32")[0], "o")
    accept = [m, 0, 1, m // 2, -3, m + 5]
    acc = torch.tensor(accept, dtype=torch.int32, device="cuda")
    o2 = binding.lin_decode_multi(*d, gd, S, accept=acc, scale=0.4)
    assert torch.equal(o, o2)
    S3 = dev(S0)
    assert binding.lin_decode_multi(*d, gd, S3, accept=acc, want_output=False) is None
    assert torch.equal(S, S3)
    for n, a in enumerate(min(max(a, 0), m) for a in accept):
        r = slice(n * m, n * m + a)
        _, rS, _, A = lin(q[r], k[r], v[r], g if fixed else g[r], S0[n:n + 1], 0.4)
        es = token_bounds((ro, rS), ao, A, dk, m, "f32")[1] if a else 0.0
        close(S[n:n + 1], rS, es, f"S of {a}")


def test_step_strides_and_values_that_are_not_finite():
    import torch
    from gated_delta_rule_59_amd import binding
    N, Hk, H, dk, dv = 4, 2, 4, 64, 128
    q, k, v, g, S0 = make((22, 1), N, Hk, H, dk, dv, N)
    fused = torch.zeros(N, 2 * Hk * dk + H * dv, device="cuda", dtype=torch.bfloat16)
    qv, kv = fused[:, :Hk * dk].view(N, Hk, dk), fused[:, Hk * dk:2 * Hk * dk].view(N, Hk, dk)
    vv = fused[:, 2 * Hk * dk:].view(N, H, dv)
    qv.copy_(dev(q, "bf16")), kv.copy_(dev(k, "bf16")), vv.copy_(dev(v, "bf16"))
    S, S2 = dev(S0), dev(S0)
    o = binding.lin_decode_step(qv, kv, vv, dev(g), S)
    o2 = binding.lin_decode_step(qv.contiguous(), kv.contiguous(), vv.contiguous(), dev(g), S2)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    vv[1, 2, 3] = float("nan")
    S2 = dev(S0)
    o3 = binding.lin_decode_step(qv, kv, vv, dev(g), S2)
    bad = torch.isnan(o3)
    assert bad[1, 2, 3] and bad.sum() == 1 and torch.equal(o3[~bad], o[~bad])
    bad = torch.isnan(S2)
    assert bad[1, 2, :, 3].all() and bad.sum() == dk and torch.equal(S2[~bad], S[~bad])


def test_a_prompt_and_its_tokens_agree():
    """A prompt, then tokens one by one, against the whole prompt."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((23, 1), 140, 2, 4, 128, 128, 1)
    ro, rS, ao, A = lin(q, k, v, g, S0, 1.0)
    eo, es = bounds((ro, rS), ao, A, 128, 140, "f32")
    d = [dev(a, "bf16") for a in (q, k, v)]
    gd = dev(g)
    _, S = binding.lin_chunk_fwd(*[t[None, :130] for t in d], gd[None, :130], dev(S0))
    o = torch.cat([binding.lin_decode_step(*[t[i:i + 1] for t in d], gd[i:i + 1], S) for i in range(130, 140)])
    close(o, ro[130:], eo[130:], "o")
    close(S, rS, es, "S")


def test_refusals_of_tensors():
    import torch
    from gated_delta_rule_59_amd import binding
    z = torch.zeros(2, 3, 2, 64, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(2, 3, 2, device="cuda")
    S = torch.zeros(2, 2, 64, 64, device="cuda")
    for bad, kind in ((lambda: binding.lin_chunk_fwd(z, z, z.float(), g), TypeError),
                      (lambda: binding.lin_chunk_fwd(z, z[:, :2], z, g), ValueError),
                      (lambda: binding.lin_chunk_fwd(z, z[:, :, :1], z, g), ValueError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g[:, :, :1]), ValueError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g.double()), TypeError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g.cpu()), ValueError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g, S[:1]), ValueError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g, S.bfloat16()), TypeError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g, out_dtype=torch.float16), TypeError),
                      (lambda: binding.lin_chunk_fwd(z, z, z, g, o=torch.zeros(2, 3, 2, 32, device="cuda")), ValueError),
                      (lambda: binding.lin_decode_step(z, z, z, g, S), ValueError),
                      (lambda: binding.lin_decode_multi(z, z, z, g, S.transpose(2, 3)), ValueError),
                      (lambda: binding.lin_decode_multi(z, z, z, g, S, accept=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                      (lambda: binding.lin_chunk_fwd(z[..., 1:], z[..., 1:], z, g), binding.KDAError)):
        with pytest.raises(kind):
            bad()
