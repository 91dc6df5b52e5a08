"""kda_adjust_logits against the definition in 64 bits.

Adjusted logits: at most seven operations in 32 bits, each off by 2^-24 of what it gives; what they give is
bounded by the sum of the parts' absolute values. Probabilities: with that error in the exponent, the
exponent's own rounding, e^x (2^-22) and the sum's (2^-22): relative 2^-21 + 2^-23 |x - max| + twice the
logits' error."""
import numpy as np
import pytest

from tests.step_ref import logits as plain

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(seed, N, R, V, history=40, biases=5, act="bf16"):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((3 * rng.standard_normal((N, R, V))).astype(np.float32))
    x = (x.bfloat16().float() if act == "bf16" else x).numpy()
    kw = dict(repetition=1 + rng.random(N), frequency=rng.random(N) - 0.3, presence=rng.random(N) - 0.3,
              temperature=0.3 + rng.random(N))
    kw = {k: v.astype(np.float32) for k, v in kw.items()}
    if history:
        kw.update(history=rng.integers(0, max(1, min(V, 2 * history)), (N, history)).astype(np.int32),
                  history_lens=rng.integers(0, history + 1, N).astype(np.int32),
                  prompt_lens=rng.integers(0, history + 1, N).astype(np.int32))
    if R > 1:
        kw["drafts"] = rng.integers(0, min(V, 2 * history + 2), (N, R - 1)).astype(np.int32)
    if biases:
        kw.update(bias_ids=rng.integers(0, V, (N, biases)).astype(np.int32),
                  bias=rng.standard_normal((N, biases)).astype(np.float32) * 3,
                  bias_counts=rng.integers(0, biases + 1, N).astype(np.int32))
    words = (V + 31) // 32
    kw["mask"] = (rng.integers(0, 2 ** 32, (N, R, words)) | rng.integers(0, 2 ** 32, (N, R, words))).astype(np.uint32).view(np.int32)
    return x, kw


def run(x, kw, act="bf16", out="f32", probs=False, **more):
    import torch
    from gated_delta_rule_59_amd import binding
    t = {"f32": torch.float32, "bf16": torch.bfloat16}
    d = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in kw.items()}
    y = binding.adjust_logits(torch.from_numpy(x).to(t[act]).cuda(), **d, probs=probs, out_dtype=t[out], **more)
    torch.cuda.synchronize()
    return y


def size_of(x, kw):
    """What the parts of an adjusted logit add up to in absolute values: its errors are relative to it."""
    N = x.shape[0]
    one = lambda k, d: np.abs(kw[k]).astype(np.float64) if k in kw else np.full(N, d)  # noqa: E731
    r, most = one("repetition", 1.0), float(kw["history"].shape[1] if "history" in kw else 0) + x.shape[1]
    s = np.where(np.isfinite(x), np.abs(x), 0).max((1, 2)) * np.maximum(r, 1 / np.maximum(r, 1e-9))
    s = s + one("frequency", 0.0) * most + one("presence", 0.0)
    s = s + (np.where(np.isfinite(kw["bias"]), np.abs(kw["bias"]), 0).max(1) if "bias" in kw else 0.0)
    t = one("temperature", 1.0)
    return (s / np.where(t > 0, t, 1.0))[:, None, None]


def check(x, kw, act="bf16", out="f32", **more):
    half = {"bf16": 2.0 ** -8, "f32": U}[out]
    got = run(x, kw, act, out, **more).double().cpu().numpy()
    want = plain(x, **kw)
    e = 8 * U * size_of(x, kw)
    with np.errstate(invalid="ignore"):
        fine = np.isfinite(want)
        assert (np.isnan(got) == np.isnan(want)).all() and (got[~fine & ~np.isnan(want)] == want[~fine & ~np.isnan(want)]).all()
        err = np.abs(got - want)
        assert (err <= e + half * np.abs(want))[fine].all(), np.nanmax((err / (e + half * np.abs(want)))[fine])
    p = run(x, kw, act, out, probs=True, **more).double().cpu().numpy()
    q = plain(x, **kw, probs=True)
    assert (np.isnan(p) == np.isnan(q)).all()
    with np.errstate(invalid="ignore"):
        top = np.nanmax(np.where(np.isfinite(want), want, -np.inf), -1, keepdims=True, initial=-1e30)
        far = np.where(np.isfinite(want) & (top > -1e30), np.abs(want - top), 0)
        bound = (half + 2.0 ** -21 + 2.0 ** -23 * far + 2 * e) * np.abs(q) + 2.0 ** -126
        ok = (np.abs(p - q) <= bound) | np.isnan(q)
    assert ok.all(), (np.argwhere(~ok)[:3], p[~ok][:3], q[~ok][:3])
    return want, q


@pytest.mark.parametrize("N,R,V,act,out", [
    (1, 1, 1, "f32", "f32"), (2, 1, 7, "bf16", "bf16"), (3, 3, 33, "bf16", "f32"), (1, 5, 4095, "f32", "f32"),
    (2, 2, 4096, "bf16", "f32"), (5, 1, 4097, "f32", "bf16"), (7, 4, 12289, "bf16", "f32"), (3, 1, 50257, "f32", "f32"),
    (2, 3, 131072, "bf16", "f32"), (300, 3, 9001, "bf16", "f32"), (1, 40, 100, "bf16", "f32")])
def test_against_definition(N, R, V, act, out):
    print(f"logits {N}x{R}x{V} {act}->{out}", flush=True)
    check(*make((81, N, R, V), N, R, V, act=act), act=act, out=out)


@pytest.mark.parametrize("gone", ["history", "drafts", "bias", "mask", "temperature", "repetition", "frequency",
                                  "presence", "prompt_lens", "bias_counts", "all"])
def test_without(gone):
    x, kw = make((82, 1), 4, 3, 5000)
    groups = dict(history=("history", "history_lens", "prompt_lens"), bias=("bias", "bias_ids", "bias_counts"))
    for k in (list(kw) if gone == "all" else groups.get(gone, (gone,))):
        del kw[k]
    check(x, kw)


def test_long_histories_count():
    """One token thousands of times, ids that are no tokens, prompts and drafts that overlap."""
    x, kw = make((83, 1), 3, 4, 6000, history=20000)
    kw["history"][0] = 17
    kw["history"][1, ::3] = [-1, 6000, 2 ** 31 - 1, -2 ** 31][1]
    kw["history"][2, :9000] = np.arange(9000) % 7000
    kw["history_lens"][:] = [20000, 19999, 30000]
    kw["prompt_lens"][:] = [100, -5, 40000]
    kw["drafts"][0] = [17, 17, 5999]
    kw["drafts"][1] = [-1, 6000, 5999]
    check(x, kw)


def test_the_last_bias_of_a_token_counts():
    x, kw = make((84, 1), 3, 2, 300, biases=200)
    kw["bias_ids"][:] = kw["bias_ids"] % 40
    kw["bias_ids"][0, 5], kw["bias_ids"][0, 6] = -1, 300
    kw["bias_counts"][:] = [200, 1, 999]
    check(x, kw)


def test_rows_that_nothing_is_left_of():
    x, kw = make((85, 1), 4, 2, 5000)
    kw["mask"][0] = 0
    kw["mask"][1, 1] = 0
    kw["mask"][1, 1, 156] = 1 << 6   # one token, in the last block
    kw["mask"][2, 0] = 0
    kw["mask"][2, 0, 156] = np.int32(-1) ^ 0xff  # bits past the vocabulary are no tokens
    kw["temperature"][3] = 0
    kw["mask"][3, 0] = 0
    _, p = check(x, kw)
    assert (p[0] == 0).all() and p[1, 1, 4998] == 1.0 and (p[2, 0] == 0).all() and (p[3, 0] == 0).all()


def test_values_that_are_not_finite():
    """Masked ones do not count; NaN, infinities and the type's lowest values that do."""
    x, kw = make((86, 1), 9, 1, 5000, act="f32")
    for k in ("repetition", "frequency", "presence", "bias", "bias_ids", "bias_counts"):
        del kw[k]
    off = (kw["mask"].view(np.uint32)[:, 0, np.arange(5000) // 32] >> (np.arange(5000) % 32)) & 1 == 0
    for n in range(3):
        x[n, 0, off[n]] = [np.nan, np.inf, -np.inf][n]
    on = [np.flatnonzero(~o) for o in off]
    x[3, 0, on[3][4000 % len(on[3])]] = np.nan
    x[4, 0, on[4][[5, 4000 % len(on[4])]]] = np.inf
    x[5, 0, on[5][:3000]] = -np.inf
    x[6, 0, on[6][1:]] = np.finfo(np.float32).min
    x[7, 0] = np.finfo(np.float32).min
    x[8, 0, on[8][3]], x[8, 0, on[8][9]] = np.nan, np.inf
    kw["temperature"][7] = 1.0
    check(x, kw, act="f32")
    kw["temperature"][:] = 0.0
    kw["temperature"][1], kw["temperature"][2] = -1.0, np.nan
    check(x, kw, act="f32")


def test_the_first_of_equal_ones():
    """Greedy rows whose largest value comes several times, within a block, across blocks and lanes."""
    x = np.zeros((4, 1, 20000), np.float32)
    x[0, 0, [19999, 4096, 4095, 12000]] = 5
    x[1, 0, [9001, 9000, 9300]] = 5
    x[3] = -np.inf
    kw = dict(temperature=np.zeros(4, np.float32))
    _, p = check(x, kw, act="f32")
    assert p[0, 0, 4095] == 1 and p[1, 0, 9000] == 1 and p[2, 0, 0] == 1 and (p[3] == 0).all()


def test_extreme_temperatures():
    x, kw = make((87, 1), 4, 1, 3000, act="f32")
    kw["temperature"][:] = [1e-3, 1e4, 1e-30, 1e30]
    check(x, kw, act="f32")


def test_infinite_biases():
    """A bias that bans or forces a token holds for tokens of the history and drafts too."""
    x, kw = make((89, 1), 4, 3, 5000, biases=6)
    kw["bias_ids"][:] = np.arange(6) * 3
    kw["bias"][:, ::2] = -np.inf
    kw["bias"][3, 1] = np.inf
    kw["bias_counts"][:] = 6
    kw["history"][0, :6] = np.arange(6) * 3
    kw["history"][3, 5] = 3
    kw["history_lens"][:] = 40
    kw["prompt_lens"][:] = [0, 40, 20, 3]
    kw["drafts"][1] = [6, 12]
    kw["mask"][:, :, 0] = -1
    _, p = check(x, kw)
    assert (p[:, :, [0, 6, 12]] == 0).all() and (p[3, :, 3] == 1).all()


def test_infinite_temperatures():
    """What is allowed shares the row evenly; what is masked, and the end of the last block, stay out."""
    x, kw = make((90, 1), 3, 2, 5000)
    kw["temperature"][:] = np.inf
    kw["mask"][0] = -1
    p = run(x, kw, probs=True).double().cpu().numpy()
    y = run(x, kw).double().cpu().numpy()
    on = (kw["mask"].view(np.uint32)[:, :, np.arange(5000) // 32] >> (np.arange(5000) % 32)) & 1 == 1
    assert (p[~on] == 0).all() and (y[~on] == -np.inf).all() and (np.abs(y[on]) < 1e-35).all()
    assert (np.abs(p * on.sum(-1, keepdims=True) - 1)[on] <= 2.0 ** -20).all()


def test_in_place_and_strided():
    import torch
    from gated_delta_rule_59_amd import binding
    x, kw = make((88, 1), 3, 2, 1001)
    want, p = plain(x, **kw), plain(x, **kw, probs=True)
    d = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    for probs in (False, True):
        fresh = run(x, kw, probs=probs, out="bf16")
        wide = torch.full((3, 2, 1040), 9.0, dtype=torch.bfloat16, device="cuda")
        view = wide[:, :, 3:1004]
        view.copy_(torch.from_numpy(x))
        assert binding.adjust_logits(view, **d, probs=probs, out=view) is view
        assert torch.equal(view, fresh) and (wide[:, :, :3] == 9).all() and (wide[:, :, 1004:] == 9).all()
        # rows outermost
        turned = torch.empty(2, 3, 1001, device="cuda").transpose(0, 1)
        binding.adjust_logits(torch.from_numpy(x).cuda(), **d, probs=probs, out=turned)
        assert torch.equal(turned, run(x, kw, act="f32", probs=probs))
        # fp32 in place, rows outermost
        y = torch.from_numpy(x).cuda().transpose(0, 1).contiguous().transpose(0, 1)
        assert binding.adjust_logits(y, **d, probs=probs, out=y) is y
        assert torch.equal(y, run(x, kw, act="f32", probs=probs))
    # one mask for all rows, a wide history
    kw["mask"] = kw["mask"][:1, :1]
    d["mask"] = torch.from_numpy(kw["mask"].copy()).cuda().expand(3, 2, -1)
    big = torch.full((3, 77), 5, dtype=torch.int32, device="cuda")
    big[:, 7:47].copy_(d["history"])
    d["history"] = big[:, 7:47]
    got = binding.adjust_logits(torch.from_numpy(x).bfloat16().cuda(), **d)
    kw["mask"] = np.broadcast_to(kw["mask"], (3, 2, kw["mask"].shape[-1]))
    assert torch.equal(got, run(x, kw))


def test_refusals_of_tensors():
    import torch
    from gated_delta_rule_59_amd import binding
    x = torch.zeros(2, 3, 100, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    for kw, kind in ((dict(history=i(2, 5)), ValueError), (dict(prompt_lens=i(2)), ValueError),
                     (dict(history=i(3, 5), history_lens=i(2)), ValueError),
                     (dict(history=i(2, 5).long(), history_lens=i(2)), TypeError),
                     (dict(drafts=i(2, 3)), ValueError), (dict(repetition=f(3)), ValueError),
                     (dict(presence=f(2).double()), TypeError), (dict(bias=f(2, 3)), ValueError),
                     (dict(bias=f(2, 3), bias_ids=i(2, 4)), ValueError), (dict(bias_counts=i(2)), ValueError),
                     (dict(mask=i(2, 3, 3)), ValueError), (dict(mask=f(2, 3, 4)), TypeError),
                     (dict(temperature=f(2).cpu()), ValueError), (dict(out=f(2, 3, 99)), ValueError),
                     (dict(out_dtype=torch.float16), TypeError)):
        with pytest.raises(kind):
            binding.adjust_logits(x, **kw)
    with pytest.raises(ValueError):
        binding.adjust_logits(x.transpose(1, 2))
    with pytest.raises(binding.KDAError):
        binding.adjust_logits(x, probs=True, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.KDAError):
        binding.adjust_logits(x, out=torch.zeros(2, 1, 100, device="cuda").expand(2, 3, 100))
    empty = dict(history=i(2, 0), history_lens=i(2), bias=f(2, 0), bias_ids=i(2, 0))
    assert torch.equal(binding.adjust_logits(x, **empty), x)
