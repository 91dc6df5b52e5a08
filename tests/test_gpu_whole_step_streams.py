"""What verification of drafts through linear attention allocates, and where. (It takes new streams: see
test_gpu_whole_step.py, beside which it runs.)"""
import pytest

from tests.test_gpu_lin import dev, make
from tests.test_gpu_streams import Allocations

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("commit", [False, True])
def test_lin_decode_multi_allocates_its_result_on_the_given_stream(commit):
    import torch
    from gated_delta_rule_59_amd import binding
    N, m = 3, 5
    q, k, v, g, S0 = make((43, 1), N * m, 1, 2, 64, 64, N)
    d = [dev(x, "bf16").view(N, m, *x.shape[1:]) for x in (q, k, v)] + [dev(g).view(N, m, 2)]
    accept = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda") if commit else None
    S = dev(S0)
    want = binding.lin_decode_multi(*d, S, accept=accept)
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current in (torch.cuda.current_stream(), other):
        with torch.cuda.stream(current):
            for stream in (s, None, current):
                S2 = dev(S0)
                torch.cuda.synchronize()
                with Allocations() as at:
                    got = binding.lin_decode_multi(*d, S2, accept=accept, stream=stream)
                assert at.streams == [(stream or current).cuda_stream]
                torch.cuda.synchronize()
                assert torch.equal(got, want) and torch.equal(S2, S)
                with Allocations() as at:
                    binding.lin_decode_multi(*d, S2, accept=accept, stream=stream, o=got)
                assert at.streams == []
                torch.cuda.synchronize()
