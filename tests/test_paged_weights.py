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
