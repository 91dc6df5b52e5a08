"""kda_page_plan against the definition, one sequence after the other: whole numbers, equal."""
import numpy as np
import pytest

from tests.step_ref import plan

pytestmark = pytest.mark.gpu


def run(table, held, lens, new_lens, free, ring, page_size, max_tokens, **kw):
    import torch
    from gated_delta_rule_59_amd import binding
    i32 = lambda x: torch.from_numpy(np.array(x, np.int64).astype(np.int32)).cuda()  # noqa: E731
    t, f = i32(table), i32(free)
    state = [i32(x) for x in (held, lens, new_lens)]
    r = i32(ring)
    out = binding.page_plan(t, *state, f, r, page_size=page_size, max_tokens=max_tokens, **kw)
    torch.cuda.synchronize()
    for x, was in zip((*state, r), (held, lens, new_lens, ring)):
        assert (x.cpu().numpy() == np.array(was)).all()
    got = dict(zip(("held", "ring", "seq_lens", "cu", "slots", "positions"), out), table=t, free=f)
    return {k: v.cpu().numpy() for k, v in got.items()}


def check(*args, **kw):
    got, want = run(*args, **kw), plan(np.array(args[0]), *args[1:4], np.array(args[4]), *args[5:])
    for k in want:
        assert (got[k] == want[k]).all(), (k, np.flatnonzero((got[k] != want[k]).ravel())[:5])
    return want


def make(seed, N, page, hi, new, ending=0, spare=None, waiting=0.2, extra=0.2):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi + 1, N)
    fresh = rng.integers(1, 2 * new, N) * (rng.random(N) >= waiting)
    fresh[rng.permutation(N)[:ending]] = -1 - rng.integers(0, 5)
    held = -(-lens // page)
    held += (rng.random(N) < extra) & (held > 0)
    width = (hi + 2 * new) // page + 2
    used = int(held.sum())
    need = np.maximum(0, -(-(lens + np.maximum(fresh, 0)) // page) - held)[fresh >= 0].sum()
    spare = int(need) + 3 if spare is None else int(need * spare)
    ids = rng.permutation(used + spare)
    table = -np.ones((N, width), np.int64)
    table[np.arange(width)[None] < held[:, None]] = ids[:used]
    cap = used + spare + 1
    free = -np.ones(cap, np.int64)
    head = int(rng.integers(0, cap))
    free[(head + np.arange(spare)) % cap] = ids[used:]
    return table, held, lens, fresh, free, [head, spare], page


@pytest.mark.parametrize("N,page,hi,new,ending", [
    (1, 16, 100, 1, 0), (1, 1, 0, 1, 0), (3, 20, 50, 4, 1), (64, 64, 5000, 1, 3), (255, 16, 300, 40, 20),
    (256, 1, 50, 3, 30), (257, 48, 900, 7, 100), (1023, 8, 100, 2, 5), (1024, 16, 100, 2, 0), (1025, 16, 64, 9, 300),
    (3000, 7, 30, 5, 1000), (40, 256, 100000, 3000, 2)])
def test_against_definition(N, page, hi, new, ending):
    print(f"plan N={N} page={page} hi={hi} new={new} ending={ending}", flush=True)
    args = make((71, N, page), N, page, hi, new, ending)
    total = int(np.maximum(args[3], 0).sum())
    want = check(*args, max(1, total))
    assert want["cu"][-1] == total
    check(*args, max(1, total) + 700)


@pytest.mark.parametrize("spare", [0.0, 0.3, 0.9])
@pytest.mark.parametrize("N", [30, 1500])
def test_pages_that_do_not_suffice(N, spare):
    args = make((72, N), N, 16, 200, 30, N // 10, spare=spare)
    want = check(*args, int(np.maximum(args[3], 0).sum()) + 1)
    assert want["cu"][-1] < np.maximum(args[3], 0).sum()


@pytest.mark.parametrize("N", [30, 1500])
def test_tokens_that_do_not_fit(N):
    args = make((73, N), N, 16, 200, 30, N // 10)
    check(*args, int(np.maximum(args[3], 0).sum()) // 2 + 1)
    check(*args, 1)


def test_everyone_ends_and_no_one_asks():
    table, held, lens, fresh, free, ring, page = make((74, 1), 50, 16, 500, 4)
    want = check(table, held, lens, np.full(50, -1), free, ring, page, 64)
    assert (want["held"] == 0).all() and (want["slots"] == -1).all() and want["ring"][1] == ring[1] + held.sum()
    check(table, held, lens, np.zeros(50, int), free, ring, page, 64)


def test_a_ring_with_no_room_loses_pages():
    check(np.arange(12).reshape(3, 4), [4, 4, 4], [3, 3, 3], [-1, 1, -1], np.arange(20, 25), [3, 2], 4, 8)
    check(np.arange(12).reshape(3, 4), [4, 4, 4], [3, 3, 3], [-1, -1, -1], np.arange(20, 25), [4, 5], 4, 8)


def test_pages_that_come_back_are_for_the_next_call():
    check([[5, 6], [-1, -1]], [2, 0], [8, 0], [-1, 3], [0, 0, 0], [0, 0], 4, 8)


def test_values_out_of_range():
    table = np.arange(40).reshape(5, 8)
    table[2, 1] = -7
    check(table, [-3, 99, 2, 8, 0], [5, -4, 7, 2 ** 31 - 1, 2 ** 31 - 5], [2, 3, 1, 9, 2], np.arange(50, 60), [-4, 99], 4, 20)
    check(table, [1, 1, 1, 1, 1], [1] * 5, [2 ** 31 - 1] * 5, np.arange(50, 60), [2 ** 31 - 1, 4], 4, 20)
    check(table, [0] * 5, [0] * 5, [3] * 5, np.arange(50, 60), [25, -1], 4, 20)


def test_long_positions():
    """Tables that reach 2^31 - 1 tokens, in pages of 2^20."""
    table = np.arange(2 * 2048).reshape(2, 2048)
    check(table, [2047, 2048], [2 ** 31 - 2 ** 20 - 3, 2 ** 31 - 10], [6, 9], np.arange(9000, 9004), [1, 2], 2 ** 20, 16)


def test_strided_table_and_given_outputs():
    import torch
    from gated_delta_rule_59_amd import binding
    args = make((75, 1), 33, 16, 300, 5, 4)
    want = plan(*args, 200)
    i32 = lambda x: torch.from_numpy(np.array(x, np.int64).astype(np.int32)).cuda()  # noqa: E731
    table, held, lens, fresh, free, ring, page = args
    wide = torch.full((33, table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    t = wide[:, 4:4 + table.shape[1]]
    t.copy_(i32(table))
    outs = dict(held_out=torch.empty(33, dtype=torch.int32, device="cuda"), ring_out=torch.empty(2, dtype=torch.int32, device="cuda"),
                seq_lens=torch.empty(33, dtype=torch.int32, device="cuda"), cu_seqlens=torch.empty(34, dtype=torch.int32, device="cuda"),
                slots=torch.empty(200, dtype=torch.int64, device="cuda"), positions=torch.empty(200, dtype=torch.int32, device="cuda"))
    got = binding.page_plan(t, i32(held), i32(lens), i32(fresh), i32(free), i32(ring), page_size=page, max_tokens=200, **outs)
    for x, y, name in zip(got, outs.values(), ("held", "ring", "seq_lens", "cu", "slots", "positions")):
        assert x is y and (x.cpu().numpy() == want[name]).all(), name
    assert (t.cpu().numpy() == want["table"]).all() and (wide[:, :4] == -5).all() and (wide[:, -5:] == -5).all()


def test_refusals_of_tensors():
    import torch
    from gated_delta_rule_59_amd import binding
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ok = [i(4, 6), i(4), i(4), i(4), i(9), i(2)]
    for at, bad, kind in ((0, i(4, 6).long(), TypeError), (0, i(6, 4).t(), ValueError), (1, i(5), ValueError),
                          (2, i(4).cpu(), ValueError), (3, i(8)[::2], ValueError), (5, i(3), ValueError)):
        with pytest.raises(kind):
            binding.page_plan(*ok[:at], bad, *ok[at + 1:], page_size=4, max_tokens=8)
    for kw in (dict(page_size=0, max_tokens=8), dict(page_size=4, max_tokens=0), dict(page_size=4, max_tokens=8, held_out=ok[1])):
        with pytest.raises(binding.KDAError):
            binding.page_plan(*ok, **kw)
    with pytest.raises(TypeError):
        binding.page_plan(*ok, page_size=4, max_tokens=8, slots=i(8))
