"""libkda: Kimi Delta Attention (KDA) chunked prefill and decode on AMD MI355X (gfx950), and the calls of a serving
step around them.

The computation lives in the HIP kernels of csrc/, behind the C ABI declared in
include/kda.h; `binding` marshals torch tensors into it. `inputs` makes the seeded
synthetic workloads. Importing the package does not load the library; the first call does,
and fails loudly if it has not been built (python -m gated_delta_rule_59_amd.build).
"""
__all__ = ["chunk_fwd", "chunk_fwd_noalloc", "chunk_fwd_workspace_bytes", "decode_step", "decode_multi", "check_gates",
           "kv_append", "paged_decode", "paged_decode_workspace_bytes", "verify_drafts", "lin_chunk_fwd",
           "lin_chunk_fwd_workspace_bytes", "lin_decode_step", "lin_decode_multi", "page_plan", "adjust_logits"]


def __getattr__(name):
    if name in __all__:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
