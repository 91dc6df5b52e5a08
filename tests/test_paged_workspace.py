"""The workspace that kda_paged_decode and kda_verify_drafts ask for (host only)."""
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


def test_a_window_or_a_shorter_bound_needs_no_more(b):
    """One workspace, sized with window = 0 and the longest max_len, serves every layer of a stack."""
    rng = random.Random(5)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731

    def need(N, m, Hq, Hkv, d, dtype, page, max_pages, max_len, window):
        a = b.PagedDecodeArgs()
        a.N, a.m, a.Hq, a.Hkv, a.d = N, m, Hq, Hkv, d
        a.act_dtype = a.out_dtype = 0 if dtype == 0 else 1
        a.cache.dtype, a.cache.num_pages, a.cache.page_size, a.cache.max_pages = dtype, 9, page, max_pages
        a.max_len, a.window, a.scale = max_len, window, 1.0
        return b.lib().kda_paged_decode_workspace_bytes(ctypes.byref(a))

    more = 0
    for _ in range(20000):
        Hkv, page, max_len = log(1, 64), log(1, 512), log(1, 300000)
        shape = (log(1, 5000), log(1, 64), Hkv * log(1, 16), Hkv, rng.choice([32, 64, 128]),
                 rng.choice([0, 1, 2]), page, -(-max_len // page))
        full = need(*shape, max_len, 0)
        assert full != b.SIZE_MAX
        with_window = need(*shape, max_len, log(1, 400000))
        assert with_window <= full and need(*shape, rng.randint(1, max_len), 0) <= full
        more += with_window < full
    assert more > 1000


def test_verification_is_limited_by_its_launches(b):
    """Sequences times blocks of 1024 tokens are no limit of the launches, which have a wave per sequence,
    or at most 65,536 waves, in whole workgroups of 256."""
    def need(N, V):
        a = b.VerifyArgs()
        a.N, a.m, a.V, a.dtype = N, 4, V, 1
        return b.lib().kda_verify_drafts_workspace_bytes(ctypes.byref(a))

    assert need(1 << 15, 1 << 20) == 1 << 29       # 32,768 sequences over 2^20 tokens
    assert need(1, 1 << 30) == 1 << 24
    most = 4 * ((2 ** 32 - 1) // 256)               # four sequences to a workgroup of 256
    assert need(most, 1) == 16 * most and need(most + 1, 1) == b.SIZE_MAX
    assert need(1, (1 << 30) + 1) == b.SIZE_MAX
