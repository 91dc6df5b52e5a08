"""What the package itself offers."""
import os

import pytest

CALLS = ["chunk_fwd", "chunk_fwd_noalloc", "decode_step", "decode_multi", "check_gates", "kv_append", "paged_decode",
         "verify_drafts", "lin_chunk_fwd", "lin_decode_step", "lin_decode_multi", "page_plan", "adjust_logits"]


@pytest.mark.parametrize("name", CALLS)
def test_calls_are_reached_through_the_package(name):
    import gated_delta_rule_59_amd as kda
    from gated_delta_rule_59_amd import binding
    assert getattr(kda, name) is getattr(binding, name) and name in kda.__all__


def test_the_package_offers_nothing_that_the_binding_lacks():
    import gated_delta_rule_59_amd as kda
    from gated_delta_rule_59_amd import binding
    assert all(callable(getattr(binding, name)) for name in kda.__all__)
    with pytest.raises(AttributeError):
        kda.no_such_call


def test_the_readme_names_them():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        text = f.read()
    assert all(f"`{name}`" in text for name in CALLS)
