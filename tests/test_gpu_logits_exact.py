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
