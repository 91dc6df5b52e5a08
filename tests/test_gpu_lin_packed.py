"""Packed prompts of linear attention: orders of work, and offsets that overlap."""
import numpy as np
import pytest

from tests.step_ref import lin
from tests.test_gpu_lin import bounds, close, dev, make, prompt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,most,long", [(60, 5, 70, 0), (40, 8, 60, 700), (64, 9, 40, 0), (50, 12, 30, 2000), (3, 100, 500, 900)])
def test_more_workgroups_than_places(N, H, most, long, act):
    """Up to 64 sequences with 257 .. 512 workgroups' work (the second half of them goes backwards) and with
    more, some of them in several segments."""
    lengths = [int(x) for x in np.random.default_rng((14, N, H)).integers(0, most + 1, N)]
    lengths[N // 3] = max(lengths[N // 3], long)
    print(f"lin packed {N} x {H} of up to {most} and {long} {act}", flush=True)
    prompt(make((15, N, H), sum(lengths), 1, H, 32, 32, N, act), lengths, act=act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 64, 65, 300])
def test_several_long_ones_among_short_ones(N, act):
    """States in the workspace are numbered over the sequences that have some there."""
    lengths = [int(x) for x in np.random.default_rng((16, N)).integers(0, 12, N)]
    for n, length in ((0, 700), (N // 2, 300), (N // 2 + 1, 129), (N - 1, 1025)):
        lengths[n] = length
    print(f"lin packed {N} with long ones {act}", flush=True)
    prompt(make((17, N), sum(lengths), 1, 1, 64, 32, N, act), lengths, act=act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("N,T", [(6, 1000), (64, 1000), (65, 1000), (200, 3000), (6, 200)])
def test_sequences_before_offsets_overlap_are_done(N, T, act):
    """Offsets that give tokens to many sequences: those before them keep their results, and the rows of none but
    sequences are written."""
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = make((18, N, T), T, 1, 1, 32, 32, N, act)
    cu = np.full(N + 1, 10)
    cu[0], cu[1], cu[2] = 0, 10, 160
    cu[3::2], cu[4::2] = 170, T - 5
    print(f"lin overlapping offsets {N} {T} {act}", flush=True)
    o = torch.full((1, T, 1, 32), 7.0, device="cuda")
    o, S = binding.lin_chunk_fwd(*[dev(a, act)[None] for a in (q, k, v)], dev(g)[None], dev(S0),
                                 torch.tensor(cu, dtype=torch.int32, device="cuda"), o=o)
    torch.cuda.synchronize()
    ro, rS, ao, A = lin(q[:170], k[:170], v[:170], g[:170], S0[:3], 1.0, [10, 150, 10])
    eo, es = bounds((ro, rS), ao, A, 32, 150, "f32")
    close(o[0, :170], ro, eo, "o")
    close(S[:3], rS, es, "S")
    assert (o[0, T - 5:] == 7.0).all()
