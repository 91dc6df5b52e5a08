"""The calls around a step's layers together with those of the step: prompts, then speculative steps, from
request lengths to tokens; then the calls on given streams, at the same time, and captured."""
import numpy as np
import pytest

from tests.paged_ref import attend, attend_bound, verify
from tests.step_ref import lin, logits as plain_logits, plan
from tests.test_gpu_lin import bounds, close, dev, make as make_lin, token_bounds
from tests.test_gpu_logits import make as make_logits
from tests.test_gpu_page_plan import make as make_plan
from tests.test_gpu_streams import Allocations

pytestmark = pytest.mark.gpu


def test_prompts_and_speculative_steps():
    """Five sequences: prompts through page_plan, kv_append and lin_chunk_fwd; then three steps of three drafts
    each: page_plan, kv_append, paged_decode, lin_decode_multi, adjust_logits, verify_drafts and the
    commit. One sequence ends on the way and another takes its place."""
    import torch
    from gated_delta_rule_59_amd import binding
    rng = np.random.default_rng(101)
    N, m, page, width, Hq, Hkv, d, V = 5, 3, 8, 12, 4, 2, 64, 700
    H, dk, dv = 2, 64, 64
    i32 = lambda x: torch.tensor(np.array(x), dtype=torch.int32, device="cuda")  # noqa: E731
    pool = N * width
    table, held = torch.full((N, width), -1, dtype=torch.int32, device="cuda"), i32([0] * N)
    free, ring = i32(rng.permutation(pool)), i32([7, pool])
    kc = torch.zeros(pool, page, Hkv, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    S = torch.zeros(N, H, dk, dv, device="cuda")
    lens = [0] * N
    keys, vals = [np.zeros((0, Hkv, d))] * N, [np.zeros((0, Hkv, d))] * N
    states = np.zeros((N, H, dk, dv))

    def planned(new):
        nonlocal held, ring
        want = plan(*(x.cpu().numpy() for x in (table, held)), lens, new, free.cpu().numpy(), ring.cpu().numpy(), page, 64)
        out = binding.page_plan(table, held, i32(lens), i32(new), free, ring, page_size=page, max_tokens=64)
        held, ring, seq_lens, cu, slots, positions = out
        got = dict(table=table, free=free, held=held, ring=ring, seq_lens=seq_lens, cu=cu, slots=slots, positions=positions)
        for k, v in got.items():
            assert (v.cpu().numpy() == want[k]).all(), k
        return seq_lens, cu, slots

    def appended(k, v, cu, slots, new):
        """Keys and values [total, Hkv, d] of the step into the cache; slots say where they are."""
        binding.kv_append(k[None], v[None], kc, vc, table, i32(lens), cu_seqlens=cu)
        total = int(cu[-1])
        assert torch.equal(kc.view(-1, Hkv, d)[slots[:total]], k) and torch.equal(vc.view(-1, Hkv, d)[slots[:total]], v)
        at = 0
        for n, x in enumerate(new):
            x = max(x, 0)
            keys[n] = np.concatenate([keys[n][:lens[n]], k[at:at + x].double().cpu().numpy()])
            vals[n] = np.concatenate([vals[n][:lens[n]], v[at:at + x].double().cpu().numpy()])
            at += x

    def prompts(new):
        _, cu, slots = planned(new)
        total = sum(max(x, 0) for x in new)
        kv = [torch.from_numpy(rng.standard_normal((total, Hkv, d)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]
        appended(*kv, cu, slots, new)
        q, k, v, g, _ = make_lin((102, total), total, 1, H, dk, dv, N)
        start = states.astype(np.float32)
        for n, x in enumerate(new):  # a place that is taken anew starts from nothing
            if x > 0:
                start[n] = 0
        S.copy_(torch.from_numpy(start))
        o, _ = binding.lin_chunk_fwd(*[dev(a, "bf16")[None] for a in (q, k, v)], dev(g)[None], S, cu, S_T=S)
        each = [max(x, 0) for x in new]
        ro, rS, ao, A = lin(q, k, v, g, start, 1.0, each)
        eo, es = bounds((ro, rS), ao, A, dk, max(each), "f32")
        close(o[0], ro, eo, "o of the prompts")
        close(S, rS, es, "S of the prompts")
        states[:] = S.double().cpu().numpy()
        for n, x in enumerate(new):
            lens[n] += max(x, 0)

    def step(new, seed):
        seq_lens, cu, slots = planned(new)
        live = [n for n in range(N) if new[n] > 0]
        kv = [torch.from_numpy(rng.standard_normal((len(live) * m, Hkv, d)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]
        appended(*kv, cu, slots, new)
        q = torch.from_numpy(rng.standard_normal((N, m, Hq, d)).astype(np.float32)).cuda().bfloat16()
        o = binding.paged_decode(q, kc, vc, table, seq_lens)
        full = [len(keys[n]) if n in live else 0 for n in range(N)]
        ks, vs = ([x[n][:full[n]] for n in range(N)] for x in (keys, vals))
        hq = q.double().cpu().numpy()
        ref, _ = attend(hq, ks, vs, [np.ones(x, bool) for x in full], full, d ** -0.5, 0)
        tol = attend_bound(hq, ks, vs, full, d ** -0.5, "bf16", ref, "f32")
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()
        # the drafts through the layer with decays, without touching its state
        lq, lk, lv, lg, _ = make_lin((103, seed), N * m, 1, H, dk, dv, N)
        view = lambda t: t.view(N, m, *t.shape[1:])  # noqa: E731
        args = [view(dev(a, "bf16")) for a in (lq, lk, lv)] + [view(dev(lg))]
        before = S.clone()
        lo = binding.lin_decode_multi(*args, S)
        assert torch.equal(S, before)
        ro, _, ao, A = lin(lq, lk, lv, lg, states, 1.0, [m] * N)
        close(lo, ro, token_bounds((ro, states), ao, A, dk, m, "f32")[0], "o of the drafts")
        # logits to probabilities to tokens
        x, kw = make_logits((104, seed), N, m + 1, V)
        kw["drafts"] = rng.integers(0, V, (N, m)).astype(np.int32)
        p = binding.adjust_logits(torch.from_numpy(x).bfloat16().cuda(), probs=True,
                                  **{k: torch.from_numpy(v).cuda() for k, v in kw.items()})
        wantp = plain_logits(x, **kw, probs=True)
        assert (np.abs(p.double().cpu().numpy() - wantp) <= 1e-4 * wantp + 1e-30).all()  # bounds: test_gpu_logits.py
        u = (0.02 * rng.random((N, m + 1))).astype(np.float32)  # so that some drafts stand
        drafts = p[:, :m].argmax(-1).int()
        accept, tokens = binding.verify_drafts(p, None, drafts, torch.from_numpy(u).cuda(), n_drafts=i32(np.maximum(new, 0)))
        a, t = verify(p.cpu().numpy(), None, drafts.cpu().numpy(), u, np.maximum(new, 0))
        assert (accept.cpu().numpy() == a).all() and (tokens.cpu().numpy() == t).all()
        # the commit
        binding.lin_decode_multi(*args, S, accept=accept, want_output=False)
        for n in range(N):
            r = slice(n * m, n * m + a[n])
            _, rS, _, A = lin(lq[r], lk[r], lv[r], lg[r], states[n:n + 1], 1.0)
            close(S[n:n + 1], rS, token_bounds((ro, rS), ao, A, dk, m, "f32")[1] if a[n] else 0.0, "S")
            lens[n] += int(a[n]) if new[n] > 0 else 0
        states[:] = S.double().cpu().numpy()
        return a

    prompts([13, 1, 24, 7, 0])
    stood = step([m, m, m, m, 0], 1)
    stood = stood + step([m, m, -1, m, 0], 2)
    lens[2] = 0
    prompts([0, 0, 9, 0, 17])
    stood = stood + step([m] * N, 3)
    assert stood.max() > 0
    planned([-1] * N)
    assert ring.cpu().tolist()[1] == pool


def calls():
    """A call of each kind: (name, what it allocates, function of keywords that gives its outputs)."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make_lin((111, 1), 3000, 1, 2, 64, 64, 1)
    d = [dev(a, "bf16")[None] for a in (q, k, v)] + [dev(g)[None]]
    S = dev(S0)
    assert binding.lin_chunk_fwd_workspace_bytes(*d, S) > 0
    yield "lin_chunk_fwd", 3, lambda **kw: binding.lin_chunk_fwd(*d, S, **kw)
    one = [a[0, :1] for a in d]
    keep, state = dev(S0), dev(S0)

    def token(**kw):
        o = binding.lin_decode_step(*one, state, **kw)
        return o, state
    yield "lin_decode_step", 1, token, lambda: state.copy_(keep)
    yield "lin_decode_multi", 1, lambda **kw: (binding.lin_decode_multi(*[a[:, :5] for a in d[:3]], d[3][:, :5].contiguous(), S, **kw),)
    table, held, lens, fresh, free, ring, page = make_plan((112, 1), 40, 16, 300, 6, 3)
    i32 = lambda x: torch.from_numpy(np.array(x, np.int64).astype(np.int32)).cuda()  # noqa: E731
    dp = [i32(x) for x in (table, held, lens, fresh, free, ring)]
    yield "page_plan", 1, lambda **kw: binding.page_plan(*dp, page_size=page, max_tokens=400, **kw)
    x, kw0 = make_logits((113, 1), 4, 3, 9000)
    dl = {a: torch.from_numpy(b).cuda() for a, b in kw0.items()}
    lx = torch.from_numpy(x).bfloat16().cuda()
    yield "adjust_logits", 2, lambda **kw: (binding.adjust_logits(lx, **dl, probs=True, **kw),)


NAMES = ["lin_chunk_fwd", "lin_decode_step", "lin_decode_multi", "page_plan", "adjust_logits"]


def call_of(name):
    for c in calls():
        if c[0] == name:
            return c[1], c[2], (c[3] if len(c) > 3 else lambda: None)


@pytest.mark.parametrize("name", NAMES)
def test_streams(name):
    """What a call allocates on a given stream is that stream's memory, and the results are the same."""
    import torch
    count, run, reset = call_of(name)
    reset()
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current in (torch.cuda.current_stream(), other):
        with torch.cuda.stream(current):
            for stream in (s, None, current):
                reset()
                torch.cuda.synchronize()
                with Allocations() as at:
                    got = run(stream=stream)
                if name != "lin_decode_multi":  # that one copies g on the current stream
                    assert at.streams == [(stream or current).cuda_stream] * count
                assert torch.cuda.current_stream() == current
                torch.cuda.synchronize()
                assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_captured(name):
    """Replays, with the program's own work and other calls between them, give what the call gives."""
    import torch
    _, run, reset = call_of(name)
    reset()
    want = [x.clone() for x in run()]
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        reset()
        for x in got:
            if name not in ("lin_decode_step",):
                x.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        reset()
        again = run()
        assert all(torch.equal(x, y) for x, y in zip(again, want))


@pytest.mark.parametrize("name", ["lin_chunk_fwd", "adjust_logits", "page_plan"])
def test_two_at_once(name):
    """Two calls on two streams at the same time, each with a workspace of its own."""
    import torch
    _, run, _ = call_of(name)
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [run(stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))


def test_the_same_bits_every_time():
    import torch
    for name in NAMES:
        _, run, reset = call_of(name)
        reset()
        want = [x.clone() for x in run()]
        for _ in range(3):
            reset()
            assert all(torch.equal(x, y) for x, y in zip(run(), want)), name
