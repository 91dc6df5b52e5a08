"""kda_adjust_logits where sequences share what is only read."""
import numpy as np
import pytest

from tests.test_gpu_logits import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,R,V", [(3, 2, 1001), (300, 3, 9001)])
@pytest.mark.parametrize("probs", [False, True])
def test_one_history_for_all_sequences(N, R, V, probs):
    """Samples of one prompt: a history expanded over the sequences, of which each counts its own length."""
    import torch
    from gated_delta_rule_59_amd import binding
    x, kw = make((91, N), N, R, V)
    kw["history"] = np.tile(kw["history"][:1], (N, 1))
    want = run(x, kw, probs=probs)
    d = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    d["history"] = d["history"][:1].contiguous().expand(N, -1)
    got = binding.adjust_logits(torch.from_numpy(x).bfloat16().cuda(), **d, probs=probs)
    assert torch.equal(got, want)


def test_one_row_of_logits_for_all():
    """Rows and sequences of logits that are the same memory, as the output's may not be."""
    import torch
    from gated_delta_rule_59_amd import binding
    x, kw = make((92, 1), 4, 3, 2000, act="f32")
    x[:] = x[:1, :1]
    one = torch.from_numpy(x[:1, :1].copy()).cuda().expand(4, 3, 2000)
    d = {k: torch.from_numpy(v).cuda() for k, v in kw.items()}
    for probs in (False, True):
        assert torch.equal(binding.adjust_logits(one, **d, probs=probs), run(x, kw, act="f32", probs=probs))
    with pytest.raises(binding.KDAError):
        binding.adjust_logits(one, out=one)
