"""kda_adjust_logits on the host: what its checks let through and what not, without a GPU (no launch is reached)."""
import pytest

from tests.test_step_api import ALIAS, BAD_SHAPE, at, b, call, logits_args  # noqa: F401


@pytest.mark.parametrize("stride,status", [(0, ALIAS), (60, ALIAS), (1, BAD_SHAPE), (59, BAD_SHAPE), (-1, BAD_SHAPE)])
def test_a_history_is_shared_or_apart(b, stride, status):  # noqa: F811
    """One that is let through meets the next check, on an output that overlaps it."""
    rc, msg = call(b, "adjust_logits", logits_args(b, history_stride=stride, out=at(2)))
    assert rc == status and msg, (rc, msg)
