"""Which launch shape the sizes of the GPU tests take, so that a change of the rules does not leave one without
tests; and that their reference has a sense of what they plant."""
import os
import subprocess

import numpy as np
import pytest

from tests.step_ref import logits as plain
from tests.test_gpu_logits import make
from tests.test_gpu_logits_large import SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    exe = tmp_path_factory.mktemp("c") / "logits_plan"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "gated_delta_rule_59_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "logits_plan.cpp"), "-o", str(exe)], check=True)

    def of(sizes):
        text = "".join("%d %d %d\n" % s for s in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    return of


def test_the_directed_tests_take_every_shape(shapes):
    want = {"small": (1, True), "large_split": (4, True), "large": (4, False)}
    for (name, (N, R, V)), (steps, blocks, splits) in zip(SHAPES.items(), shapes(SHAPES.values())):
        assert R > 1 and blocks > 2 and V % (steps * 1024), name
        assert (steps, splits == R) == want[name], name
        assert splits in (1, R)


def test_large_batches_and_single_rows(shapes):
    assert shapes([(256, 5, 131072), (1, 1, 32000), (48, 1, 32000), (49, 1, 32000), (1, 1, 1), (1, 1, 1 << 30)]) == [
        (4, 32, 1), (1, 32, 1), (1, 32, 1), (4, 8, 1), (1, 1, 1), (4, 1 << 18, 1)]


def test_the_check_notices_a_bias_that_a_draft_loses():
    """On the CPU: without the bias of a draft, or with its first entry for its last, other numbers come out."""
    x, kw = make((97, 3), 2, 3, 900, biases=3)
    kw["bias_ids"][:], kw["bias"][:], kw["bias_counts"][:] = [5, 7, 5], [9, 1, -5], 3
    kw["drafts"][:] = [5, 7]
    kw["mask"][:, :, 0] = -1   # a masked token shows nothing
    want = plain(x, **kw)
    for entry in (0, 2):
        other = dict(kw, bias_ids=kw["bias_ids"].copy())
        other["bias_ids"][:, entry] = -1
        assert (np.abs(plain(x, **other)[:, 1:, 5] - want[:, 1:, 5]) > 1).all() == (entry == 2)
