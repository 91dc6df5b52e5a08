"""The check that test_gpu_paged_weights.py makes of the attention's softmax weights tells weights of
24 bits from weights of fewer (the rounding is planted in the plain form here)."""
import numpy as np
import pytest

from tests.paged_weights import make, outside, reference, to_bf16


def fp16_parts(n):
    def rounded(w):
        rest, total = w * 2.0 ** 14, 0.0
        for _ in range(n):
            part = np.asarray(rest, np.float32).astype(np.float16).astype(np.float64)
            rest, total = rest - part, total + part
        return total * 2.0 ** -14
    return rounded


def bf16_parts(n):
    def rounded(w):
        rest, total = w, 0.0
        for _ in range(n):
            part = to_bf16(rest)
            rest, total = rest - part, total + part
        return total
    return rounded


def results(cache, out, weight):
    x = make((81, 1), cache, 40, 8, 2, 32)
    o, s = reference(*x)
    got, _ = reference(*x, weight=weight)
    return outside(to_bf16(got) if out == "bf16" else got.astype(np.float32), o, s, cache, out), got.size


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_one_fp16_part_is_seen_and_two_pass(out):
    bad, n = results("e4m3", out, fp16_parts(1))
    assert bad > n / 100
    assert results("e4m3", out, fp16_parts(2))[0] == 0


@pytest.mark.parametrize("n", [1, 2])
def test_too_few_bf16_parts_are_seen_and_three_pass(n):
    bad, size = results("bf16", "f32", bf16_parts(n))
    assert bad > size / 100
    assert results("bf16", "f32", bf16_parts(3))[0] == 0


def test_one_bf16_part_is_seen_in_bf16_results():
    """(Two are not: 2^-17 moves too few results past the edge of a bf16 step by more than the bound.)"""
    assert results("bf16", "bf16", bf16_parts(1))[0] > 0
    assert results("bf16", "bf16", bf16_parts(3))[0] == 0


@pytest.mark.parametrize("cache,rounded", [("bf16", bf16_parts(1)), ("f32", bf16_parts(1)), ("e4m3", fp16_parts(1))])
def test_a_bound_for_each_row_sees_lost_bits(cache, rounded):
    from tests import paged_rows
    rng = np.random.default_rng(83)
    lens = [2, 3, 40]
    q = to_bf16(rng.standard_normal((3, 1, 4, 64)))
    k, v = ([to_bf16(rng.standard_normal((n, 2, 64))) for n in lens] for _ in "kv")
    o, off, _, _ = paged_rows.attend_rows(q, k, v, lens, 0.01, 0, cache)
    assert not paged_rows.outside(o.astype(np.float32), o, off, "f32").any()
    got, _, _, _ = paged_rows.attend_rows(q, k, v, lens, 0.01, 0, cache, weight=rounded)
    assert paged_rows.outside(got, o, off, "f32").mean() > 0.1
