"""The workspace that kda_lin_chunk_fwd asks for (host only)."""
import ctypes
import os
import random

import pytest


@pytest.fixture(scope="module")
def b():
    from gated_delta_rule_59_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libkda not built")
    binding.lib()
    return binding


def need(b, N, T, H, dk=128, dv=128, act=1):
    a = b.LinChunkArgs()
    a.B, a.T, a.Hk, a.H, a.dk, a.dv, a.N = 1, T, H, H, dk, dv, N
    a.act_dtype, a.gate_dtype, a.out_dtype = act, 0, act
    a.cu_seqlens = 1 << 40
    return b.lib().kda_lin_chunk_fwd_workspace_bytes(ctypes.byref(a))


def test_sequences_of_one_segment_have_no_states_there(b):
    """Segments are of 128 tokens or more, and a sequence of more than one segment has at most twice as many as
    it holds whole ones; beside their states, a few bytes for each sequence and segment."""
    rng = random.Random(7)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    for _ in range(3000):
        N, T, H = log(1, 5000), log(1, 200000), log(1, 64)
        dk, dv = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        got = need(b, N, T, H, dk, dv, rng.choice([0, 1]))
        assert got != b.SIZE_MAX
        assert got <= 2 * (T // 128) * H * (dk * dv + 1) * 4 + 16 * (N + T // 128 + 2)


def test_many_short_prompts(b):
    """The states themselves are 4 bytes x 300 x 32 x 128 x 128 = 629 MB, and 6.3 GB for 3,000 prompts."""
    assert need(b, 300, 8192, 32) <= 40 << 20
    assert need(b, 3000, 60000, 32) <= 40 << 20
