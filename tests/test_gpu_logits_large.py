"""kda_adjust_logits against the definition in every launch shape and type: blocks of 1,024 tokens and of 4,096, a
row to a workgroup or all rows of a sequence, which count their drafts as they go. Bounds: test_gpu_logits.py;
that the sizes take these shapes: test_logits_plan.py."""
import numpy as np
import pytest

from tests.step_ref import logits as plain
from tests.test_gpu_logits import U, check, make, run, size_of

pytestmark = pytest.mark.gpu

SHAPES = {"small": (16, 3, 9001), "large_split": (70, 3, 9001), "large": (300, 3, 9001)}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]
shapes = pytest.mark.parametrize("shape", SHAPES)
types = pytest.mark.parametrize("act,out", TYPES)


def case(seed, shape, act, **kw):
    """The first sixteen sequences are the test's; the others, which make the batch, are alike and plain."""
    N, R, V = SHAPES[shape]
    print(f"logits {shape} {act} {seed}", flush=True)
    return make((97, seed, N), N, R, V, act=act, **kw)


def in_range(want, out):
    """Quotients beyond the result's range are infinite: -3.39e38 / 0.54 = -6.3e38 is below what 32 bits, and bf16,
    hold."""
    import torch
    y = torch.from_numpy(want).float()
    y = (y.bfloat16() if out == "bf16" else y).double().numpy()
    return np.where(np.isinf(y), y, want)


def check_in_range(x, kw, act, out):
    """As check, with the quotients that the type does not hold."""
    half = 2.0 ** -8 if out == "bf16" else U
    got, want = run(x, kw, act, out).double().cpu().numpy(), in_range(plain(x, **kw), out)
    fine = np.isfinite(want)
    assert (np.isnan(got) == np.isnan(want)).all() and (got[np.isinf(want)] == want[np.isinf(want)]).all()
    bound = 8 * U * size_of(x, kw) + half * np.abs(np.where(fine, want, 0))
    assert (np.abs(np.where(fine, got - np.where(fine, want, 0), 0)) <= bound).all()
    p, q = run(x, kw, act, out, probs=True).double().cpu().numpy(), plain(x, **kw, probs=True)
    assert (np.isnan(p) == np.isnan(q)).all()
    top = np.max(np.where(fine, want, -1e30), -1, keepdims=True)
    far = np.where(fine, np.abs(np.where(fine, want, 0) - top), 0)
    bound = (half + 2.0 ** -21 + 2.0 ** -23 * far + 16 * U * size_of(x, kw)) * np.abs(q) + 2.0 ** -126
    assert ((np.abs(p - q) <= bound) | np.isnan(q)).all()


@shapes
@types
def test_plain(shape, act, out):
    check(*case(0, shape, act), act=act, out=out)


@shapes
@pytest.mark.parametrize("gone", ["history", "drafts", "bias", "mask", "temperature", "all"])
def test_without(shape, gone):
    x, kw = case(1, shape, "bf16")
    groups = dict(history=("history", "history_lens", "prompt_lens"), bias=("bias", "bias_ids", "bias_counts"))
    for k in (list(kw) if gone == "all" else groups.get(gone, (gone,))):
        del kw[k]
    check(x, kw)


@shapes
@types
def test_drafts_of_biased_tokens(shape, act, out):
    """A draft on the way whose token has a bias: the last of several entries, an infinite one, one that the count
    leaves out; the same draft twice; drafts on both sides of the first block's end; one in the prompt only."""
    x, kw = case(2, shape, act, biases=8)
    V = x.shape[-1]
    ids = np.array([5, 4095, 5, 4096, 8999, 5, 700, 5], np.int32)
    kw["bias_ids"][:16] = ids
    kw["bias"][:16] = np.array([9, 1, 7, -2, 3, -5, np.inf, 40], np.float32)
    kw["bias_counts"][:16] = 7                     # without the last entry of token 5
    kw["history"][:16, :5] = [1023, 700, 5, 4096, 1024]
    kw["history_lens"][:16], kw["prompt_lens"][:16] = 5, [0, 5] * 8
    kw["history_lens"][8:16] = 0
    for n, d in enumerate([(5, 5), (4095, 4096), (4096, 4095), (8999, 5), (700, 700), (5, 700), (V - 1, 5), (1023, 1024)]):
        kw["drafts"][n] = kw["drafts"][n + 8] = d
    kw["bias_counts"][3] = 1
    kw["bias_counts"][11] = 8
    kw["mask"][:16, :, :] = -1
    check(x, kw, act=act, out=out)
    kw["temperature"][:16:2] = 0
    kw["bias"][:16, 6] = -np.inf
    check(x, kw, act=act, out=out)


@shapes
@types
def test_rows_that_little_is_left_of(shape, act, out):
    """Empty masks, one token, bits past the vocabulary; greedy rows among them."""
    x, kw = case(4, shape, act)
    kw["mask"][:4] = 0
    kw["mask"][1, 1, 281] = 1 << 8                         # token 9,000, the last
    kw["mask"][2, :, 281] = np.int32(-1) ^ 0x1ff           # no tokens
    kw["mask"][3, 0, 127], kw["mask"][3, 0, 128] = np.int32(-2 ** 31), 1   # tokens 4,095 and 4,096
    kw["temperature"][2:6] = 0
    kw["mask"][5, 1] = 0
    _, p = check(x, kw, act=act, out=out)
    assert (p[0] == 0).all() and p[1, 1, 9000] == 1 and (p[2] == 0).all() and (p[5, 1] == 0).all()


@shapes
@types
def test_values_that_are_not_finite(shape, act, out):
    x, kw = case(5, shape, act)
    for k in ("repetition", "frequency", "presence", "bias", "bias_ids", "bias_counts"):
        del kw[k]
    V = x.shape[-1]
    at = np.arange(V)
    low = float(np.float32(-3.3895313892515355e38)) if act == "bf16" else np.finfo(np.float32).min
    for n in range(16):
        allowed = [np.flatnonzero((kw["mask"][n, j].view(np.uint32)[at // 32] >> (at % 32)) & 1) for j in range(3)]
        for j, on in enumerate(allowed):
            off = np.setdiff1d(at, on)
            if n < 3:
                x[n, j, off] = [np.nan, np.inf, -np.inf][n]
            elif n < 6:
                x[n, j, on[5000 % len(on)]] = [np.nan, np.inf, -np.inf][n - 3]
            elif n == 6:
                x[n, j, on[[5, 4000 % len(on)]]] = np.inf
            elif n == 7:
                x[n, j, on[1:]] = low
            elif n == 8:
                x[n, j] = low
            elif n == 9:
                x[n, j] = -np.inf
            elif n == 10:
                x[n, j, on[3]], x[n, j, on[-1]] = np.nan, np.inf
    kw["temperature"][8] = 1.0
    check_in_range(x, kw, act, out)
    kw["temperature"][:16] = 0.0
    kw["temperature"][1], kw["temperature"][2] = -1.0, np.nan
    check_in_range(x, kw, act, out)


@shapes
@types
def test_the_first_of_equal_ones(shape, act, out):
    N, R, V = SHAPES[shape]
    x = np.zeros((N, R, V), np.float32)
    x[0, :, [9000, 4096, 4095, 8200]] = 5
    x[1, :, [8193, 8192, 8300]] = 5
    x[2, 0, [1023, 1024]] = x[2, 1, [3, 2]] = x[2, 2, [4097, 4100, 8999]] = 5
    x[3] = -np.inf
    x[5:] = np.arange(V) % 97 % 13
    kw = dict(temperature=np.zeros(N, np.float32))
    _, p = check(x, kw, act=act, out=out)
    assert (p[0, :, 4095] == 1).all() and (p[1, :, 8192] == 1).all() and (p[3] == 0).all() and (p[4, :, 0] == 1).all()
    assert p[2, 0, 1023] == p[2, 1, 2] == p[2, 2, 4097] == 1 and (p[5:, :, 12] == 1).all()


@shapes
@types
def test_biases_and_temperatures_without_bounds(shape, act, out):
    x, kw = case(6, shape, act, biases=6)
    kw["bias_ids"][:16] = np.array([0, 4096, 6, 8192, 12, 5000])
    kw["bias"][:16, ::2] = -np.inf
    kw["bias"][3, 1] = np.inf
    kw["bias_counts"][:16] = 6
    kw["history"][:4, :6] = kw["bias_ids"][:4]
    kw["history_lens"][:4], kw["prompt_lens"][:4] = 40, [0, 40, 20, 3]
    kw["drafts"][1], kw["drafts"][5] = [6, 12], [4096, 4096]
    kw["mask"][:16, :, 0] = -1
    kw["mask"][3, :, 128] = -1
    kw["temperature"][8:12] = [1e-3, 1e4, 1e-30, 1e30]
    _, p = check(x, kw, act=act, out=out)
    assert (p[:16, :, [0, 6, 12]] == 0).all() and (p[3, :, 4096] == 1).all()
    kw["temperature"][:16] = np.inf
    kw["bias"][3, 1] = 0
    p = run(x, kw, act=act, out=out, probs=True).double().cpu().numpy()[:16]
    at = np.arange(x.shape[-1])
    on = (kw["mask"][:16].view(np.uint32)[:, :, at // 32] >> (at % 32)) & 1 == 1
    on[:, :, [0, 6, 12]] = False
    half = 2.0 ** -8 if out == "bf16" else 0.0
    assert (p[~on] == 0).all() and (np.abs(p * on.sum(-1, keepdims=True) - 1)[on] <= 2.0 ** -20 + half).all()


@shapes
def test_long_histories_count(shape):
    x, kw = case(7, shape, "bf16", history=300, biases=40)
    kw["bias_ids"][:16] = kw["bias_ids"][:16] % 20 + 4090     # the last of several entries, across two blocks
    kw["bias_counts"][:16] = 40
    kw["history"][0] = 17
    kw["history"][1, ::3] = -1
    kw["history"][2, ::2] = 9001
    kw["history"][3] = np.arange(300) + 4000
    kw["history"][4], kw["history"][5] = 2 ** 31 - 1, -2 ** 31
    kw["history_lens"][:6], kw["prompt_lens"][:6] = [300, 299, 400, 300, 300, 300], [100, -5, 400, 200, 0, 0]
    kw["drafts"][:4] = [[17, 17], [-1, 9001], [9000, 9000], [4095, 4299]]
    check(x, kw)


@shapes
@types
def test_in_place_and_strided(shape, act, out):
    import torch
    from gated_delta_rule_59_amd import binding
    x, kw = case(8, shape, act)
    N, R, V = x.shape
    d = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    tt = {"f32": torch.float32, "bf16": torch.bfloat16}
    src = torch.from_numpy(x).to(tt[act]).cuda()
    for probs in (False, True):
        want = run(x, kw, act, out, probs=probs)
        wide = torch.full((N, R, V + 40), 9.0, dtype=tt[out], device="cuda")
        binding.adjust_logits(src, **d, probs=probs, out=wide[:, :, 3:V + 3])
        assert torch.equal(wide[:, :, 3:V + 3], want) and (wide[:, :, :3] == 9).all() and (wide[:, :, V + 3:] == 9).all()
        turned = torch.empty(R, N, V, device="cuda", dtype=tt[out]).transpose(0, 1)
        binding.adjust_logits(src, **d, probs=probs, out=turned)
        assert torch.equal(turned, want)
        if act == out:
            y = src.transpose(0, 1).contiguous().transpose(0, 1)
            assert binding.adjust_logits(y, **d, probs=probs, out=y) is y
            assert torch.equal(y, want)
