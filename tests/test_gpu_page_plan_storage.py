"""Whose memory the results of a plan are."""
import numpy as np
import pytest

from tests.test_gpu_page_plan import make

pytestmark = pytest.mark.gpu


def test_given_results_hold_nothing_else():
    """held and ring of the caller's own, which go from step to step, keep no slots and positions alive."""
    import torch
    from gated_delta_rule_59_amd import binding
    table, held, lens, fresh, free, ring, page = make((113, 1), 40, 16, 300, 6, 3)
    i32 = lambda x: torch.from_numpy(np.array(x, np.int64).astype(np.int32)).cuda()  # noqa: E731
    args = [i32(x) for x in (table, held, lens, fresh, free, ring)]
    again = [x.clone() for x in args]
    want = binding.page_plan(*args, page_size=page, max_tokens=100000)
    kept = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    got = binding.page_plan(*again, page_size=page, max_tokens=100000, held_out=kept[0], ring_out=kept[1])
    assert got[0] is kept[0] and got[1] is kept[1]
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(args, again))
    assert kept[0].untyped_storage().nbytes() == 160 and kept[1].untyped_storage().nbytes() == 8
    # where none are given: one allocation for all, and no more than its parts
    storage = want[0].untyped_storage()
    assert all(x.untyped_storage().data_ptr() == storage.data_ptr() for x in want)
    assert storage.nbytes() <= 12 * 100000 + 12 * 40 + 12 + 6 * 256
