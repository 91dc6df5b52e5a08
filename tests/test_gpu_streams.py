"""What a call allocates when a stream is given comes from that stream's memory: a block of the current
stream's may still be in use by work queued there, which the given stream does not wait for."""
import numpy as np
import pytest

from tests.paged_ref import verify

pytestmark = pytest.mark.gpu


class Allocations:
    """Streams (by address) of the device allocations made inside the with block."""

    def __enter__(self):
        import torch
        self.memory = torch.cuda.memory
        self.memory._record_memory_history(enabled="all", context=None, max_entries=1000)
        return self

    def __exit__(self, *exc):
        trace = self.memory._snapshot()["device_traces"][0]
        self.memory._record_memory_history(enabled=None)
        self.streams = [x["stream"] for x in trace if x["action"] == "alloc"]


def small(seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def append_args():
    import torch
    x = small(91)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(k=x(3, 2, 2, 64), v=x(3, 2, 2, 64), k_cache=torch.zeros(8, 16, 2, 64, device="cuda"),
                v_cache=torch.zeros(8, 16, 2, 64, device="cuda"), q=x(3, 2, 4, 64),
                block_table=torch.arange(6, **i32).view(3, 2), start=torch.tensor([0, 5, 15], **i32),
                inv_freq=torch.linspace(1, 0.01, 32, device="cuda"))


def decode_args():
    import torch
    x = small(92)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=x(2, 1, 4, 64).bfloat16(), k_cache=x(130, 16, 2, 64).bfloat16(),
                v_cache=x(130, 16, 2, 64).bfloat16(), block_table=torch.arange(130, **i32).view(2, 65),
                seq_lens=torch.tensor([1000, 777], **i32))


def verify_args():
    rng = np.random.default_rng(93)
    p = rng.random((3, 3, 20000), np.float32)
    q = rng.random((3, 2, 20000), np.float32)
    return (p / p.sum(-1, keepdims=True), q / q.sum(-1, keepdims=True),
            rng.integers(0, 20000, (3, 2)).astype(np.int32), rng.random((3, 3), np.float32))


@pytest.mark.parametrize("call", ["kv_append", "paged_decode", "verify_drafts"])
def test_serving_calls(call):
    import torch
    from gated_delta_rule_59_amd import binding
    if call == "verify_drafts":
        host = verify_args()
        dev = [torch.from_numpy(x).cuda() for x in host]
        run = lambda **kw: binding.verify_drafts(*dev, **kw)  # noqa: E731
        count = 3  # accept, tokens, workspace
    elif call == "paged_decode":
        dev = decode_args()
        assert binding.paged_decode_workspace_bytes(**dev) > 0
        run = lambda **kw: (binding.paged_decode(**dev, **kw),)  # noqa: E731
        count = 2
    else:
        dev = append_args()
        run = lambda **kw: (binding.kv_append(**dev, **kw),)  # noqa: E731
        count = 1
    want = run()
    torch.cuda.synchronize()
    if call == "verify_drafts":
        a, t = verify(*host, [2] * 3)
        assert (want[0].cpu().numpy() == a).all() and (want[1].cpu().numpy() == t).all()
    s = torch.cuda.Stream()
    other = torch.cuda.Stream()
    for current in (torch.cuda.current_stream(), other):
        with torch.cuda.stream(current):
            with Allocations() as at:
                got = run(stream=s)
            assert at.streams == [s.cuda_stream] * count
            assert torch.cuda.current_stream() == current
            with Allocations() as at:
                run()
            assert at.streams == [current.cuda_stream] * count
            with Allocations() as at:
                run(stream=current)
            assert at.streams == [current.cuda_stream] * count
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_freed_result_waits_for_the_current_stream():
    """A result of stream s that the current stream still reads: its memory goes to nobody before that."""
    import torch
    from gated_delta_rule_59_amd import binding
    dev = decode_args()
    want = binding.paged_decode(**dev)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = binding.paged_decode(**dev, stream=s)
    address = out.data_ptr()
    torch.cuda.current_stream().wait_stream(s)
    busy = torch.zeros(1 << 28, device="cuda")
    for _ in range(20):
        busy.add_(1.0)  # the copy below waits for these
    copy = out.clone()
    del out
    with torch.cuda.stream(s):
        taken = [torch.full_like(want, 7.0) for _ in range(3)]
        assert all(t.data_ptr() != address for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("call,count", [("chunk_fwd", 3), ("decode_step", 1), ("decode_multi", 1), ("check_gates", 1)])
def test_kda_calls(call, count):
    import torch
    from gated_delta_rule_59_amd import binding, inputs
    if call in ("chunk_fwd", "check_gates"):
        x = inputs.make_prefill(1, T=130, H=2)
        dev = [torch.from_numpy(a).cuda().bfloat16() for a in (x.q, x.k, x.v, x.g, x.beta)]
        S0 = torch.from_numpy(x.S0).cuda()
        if call == "chunk_fwd":
            run = lambda **kw: binding.chunk_fwd(*dev, S0, **kw)  # noqa: E731
        else:
            run = lambda **kw: (torch.tensor(binding.check_gates(dev[3], dev[4], **kw)),)  # noqa: E731
    else:
        dev = [torch.from_numpy(a).cuda().bfloat16() for a in inputs.make_decode_step(0, N=4, H=2)]
        S = torch.from_numpy(inputs.make_decode_state(4, 2)).cuda()
        if call == "decode_step":
            run = lambda **kw: (binding.decode_step(*dev, S0.copy_(S), **kw),)  # noqa: E731
            S0 = S.clone()
        else:
            run = lambda **kw: (binding.decode_multi(*[a[:, None] for a in dev], S, **kw),)  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    for current in (torch.cuda.current_stream(), other):
        with torch.cuda.stream(current):
            if call == "decode_step":  # the copy into S0 comes before the call on s
                S0.copy_(S)
                torch.cuda.synchronize()
                with Allocations() as at:
                    got = (binding.decode_step(*dev, S0, stream=s),)
            else:
                with Allocations() as at:
                    got = run(stream=s)
            assert at.streams == [s.cuda_stream] * count
            assert torch.cuda.current_stream() == current
            with Allocations() as at:
                run()
            assert at.streams == [current.cuda_stream] * count
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
