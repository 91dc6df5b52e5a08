"""kda_adjust_logits where a single bit matters: greedy ties, values of zero, biases that are added exactly."""
import numpy as np
import pytest

from tests.step_ref import logits as plain
from tests.test_gpu_logits import run

pytestmark = pytest.mark.gpu

# one workgroup per row in blocks of 1,024; all rows of a sequence to a workgroup in blocks of 4,096
SIZES = [(1, 1, 50), (2, 3, 5000), (300, 3, 9001)]


def ties(N, R, V):
    """Greedy rows of equal logits; the history and the drafts hold tokens behind the first, with no penalty."""
    x = np.zeros((N, R, V), np.float32)
    kw = dict(history=np.full((N, 3), 7, np.int32), history_lens=np.full(N, 3, np.int32),
              prompt_lens=(np.arange(N) % 4).astype(np.int32), repetition=np.full(N, 1.25, np.float32),
              temperature=np.zeros(N, np.float32))
    if R > 1:
        kw["drafts"] = np.broadcast_to(np.array([9, V - 1][:R - 1], np.int32), (N, R - 1)).copy()
    return x, kw


@pytest.mark.parametrize("N,R,V", SIZES)
def test_a_history_without_penalties_breaks_no_ties(N, R, V):
    """Zeros stay zeros, whatever the history holds: the first token of the row is chosen."""
    x, kw = ties(N, R, V)
    y = run(x, kw, act="f32").cpu().numpy()
    assert (y == 0).all()
    p = run(x, kw, act="f32", probs=True).cpu().numpy()
    assert (p[:, :, 0] == 1).all() and (p[:, :, 1:] == 0).all()


@pytest.mark.parametrize("N,R,V", SIZES)
def test_equal_biases_stay_equal(N, R, V):
    """A bias of the same value on a token that was there and on one before it that was not."""
    x, kw = ties(N, R, V)
    kw.update(bias_ids=np.broadcast_to(np.array([7, 3, 9, V - 1], np.int32), (N, 4)).copy(),
              bias=np.ones((N, 4), np.float32))
    y = run(x, kw, act="f32").cpu().numpy()
    assert (y == plain(x, **kw)).all()
    p = run(x, kw, act="f32", probs=True).cpu().numpy()
    assert (p[:, :, 3] == 1).all() and (p.sum(-1) == 1).all()


@pytest.mark.parametrize("N,R,V", SIZES)
@pytest.mark.parametrize("history", [False, True])
def test_biases_and_penalties_are_added_exactly(N, R, V, history):
    """Where the logit is zero, the result is the bias less the penalties, each rounded once: with a power of
    two for a penalty and odd last bits in the biases, the very numbers."""
    x, kw = ties(N, R, V)
    del kw["temperature"]
    bias = np.float32(1) + np.arange(1, 5, dtype=np.float32) * np.float32(2.0 ** -23)
    kw.update(bias_ids=np.broadcast_to(np.array([7, 3, 9, V - 1], np.int32), (N, 4)).copy(),
              bias=np.broadcast_to(bias, (N, 4)).copy(), frequency=np.full(N, 0.5, np.float32),
              presence=np.full(N, -0.5, np.float32))
    if not history:
        for k in ("history", "history_lens", "prompt_lens", "drafts"):
            kw.pop(k, None)
    want = plain(x, **kw)
    assert (want == want.astype(np.float32)).all()
    assert (run(x, kw, act="f32").double().cpu().numpy() == want).all()


def quotients(divisors, V):
    """Rows of logits that are products of a divisor and a 12-bit number, exact in 32 bits; the numbers."""
    rng = np.random.default_rng(95)
    q = (rng.integers(2048, 4096, (len(divisors), 1, V)) * 2.0 ** rng.integers(-14, -8, (len(divisors), 1, V)))
    q = q * rng.choice([-1.0, 1.0], q.shape)
    d = np.asarray(divisors, np.float32)
    x = q * d.astype(np.float64)[:, None, None]
    assert (x == x.astype(np.float32)).all()
    return x.astype(np.float32), q, d


DIVISORS = [1.5, 1.25, 1.125, 1.3125, 0.75, 1.75, 0.6875, 3.0, 1.0009765625, 1 / 1024]


@pytest.mark.parametrize("V", [900, 140000])
def test_temperatures_divide(V):
    """x / temperature is the quotient rounded once: the very number where there is one."""
    x, q, d = quotients(DIVISORS, V)
    y = run(x, dict(temperature=d), act="f32").double().cpu().numpy()
    assert (y == q).all(), np.argwhere(y != q)[:4]
    x = np.random.default_rng(96).standard_normal(x.shape).astype(np.float32)
    want = x.astype(np.float64) / d.astype(np.float64)[:, None, None]
    y = run(x, dict(temperature=d), act="f32").double().cpu().numpy()
    # half a step, and 2^-45 for what the second part of the reciprocal leaves
    assert (np.abs(y - want) <= 0.5 * np.spacing(np.abs(want).astype(np.float32)) + 2.0 ** -45 * np.abs(want)).all()


@pytest.mark.parametrize("V", [900, 140000])
def test_repetition_divides(V):
    """So is x / repetition, so that a greedy row chooses the first of equal ones where one of them was
    divided; x * repetition where x is below 0."""
    x, q, d = quotients(DIVISORS, V)
    N = len(d)
    x, q = np.abs(x), np.abs(q)
    x[:, 0, 1::2] *= -1
    q[:, 0, 1::2] = x[:, 0, 1::2].astype(np.float64) * d.astype(np.float64)[:, None]
    kw = dict(history=np.tile(np.arange(800, dtype=np.int32), (N, 1)), history_lens=np.full(N, 800, np.int32), repetition=d)
    y = run(x, kw, act="f32").double().cpu().numpy()
    assert (y[:, :, 800:] == x[:, :, 800:]).all()
    want, got = q[:, :, :800], y[:, :, :800]
    assert (got[:, :, ::2] == want[:, :, ::2]).all(), np.argwhere(got[:, :, ::2] != want[:, :, ::2])[:4]
    assert (np.abs(got - want) <= 0.5 * np.spacing(np.abs(want).astype(np.float32))).all()
    # token 20 is not in the history and equal to a later one's quotient
    x = np.zeros((N, 1, V), np.float32)
    most = np.float32(1 + 126 / 128)
    x[:, 0, 20], x[:, 0, 30] = most, most * d
    kw.update(history=np.full((N, 1), 30, np.int32), history_lens=np.ones(N, np.int32), temperature=np.zeros(N, np.float32))
    p = run(x, kw, act="f32", probs=True).cpu().numpy()
    assert (p[:, 0, 20] == 1).all() and (p.sum(-1) == 1).all()


def test_infinite_logits_stay_infinite():
    x = np.zeros((2, 1, 3000), np.float32)
    x[:, 0, 3::7], x[:, 0, 4::7] = np.inf, -np.inf
    kw = dict(temperature=np.array([0.7, 3.0], np.float32), repetition=np.array([1.3, 0.8], np.float32),
              history=np.tile(np.arange(3000, dtype=np.int32), (2, 1)), history_lens=np.full(2, 2000, np.int32))
    y = run(x, kw, act="f32").cpu().numpy()
    assert (y == plain(x, **kw)).all()
