"""kda_paged_decode, each result to within what its own row allows: four heads to a workgroup with a
window, with pages that are not multiples of 16 and with the head outermost; two row tiles with values
that are not finite."""
import numpy as np
import pytest

from tests.paged_rows import attend_rows, outside
from tests.test_gpu_paged_decode import make

pytestmark = pytest.mark.gpu


def run(dev, **kw):
    import torch
    from gated_delta_rule_59_amd import binding
    N, m, Hq, _ = dev["q"].shape
    lse = torch.empty((N, m, Hq), dtype=torch.float32, device="cuda")
    o = binding.paged_decode(**dev, lse=lse, **kw)
    torch.cuda.synchronize()
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(dev, h, scale, window, out):
    import torch
    got, lse = run(dev, scale=scale, window=window, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    o, off, ref, ref_off = attend_rows(h["q"], h["k"], h["v"], h["lens"], scale, window, h["cache"])
    assert not outside(got, o, off, out).any()
    seen = np.isfinite(ref)
    assert (np.isneginf(lse) == ~seen).all()
    assert (np.abs(lse[seen] - ref[seen]) <= ref_off[seen]).all()


# N, longest, m, Hq, Hkv, d, page, window, cache, result, layout
SHARED = [  # N * Hkv beyond 1024 (2048 where 32 tokens of a head are below 8 KiB): four heads to a workgroup
    (170, 300, 1, 8, 8, 64, 16, 70, "bf16", "bf16", "token"),
    (170, 300, 3, 16, 8, 64, 16, 33, "bf16", "f32", "token"),
    (300, 200, 3, 8, 8, 64, 16, 50, "e4m3", "bf16", "token"),
    (170, 300, 2, 8, 8, 32, 32, 129, "f32", "f32", "token"),
    (170, 300, 1, 8, 8, 64, 20, 0, "bf16", "bf16", "token"),
    (170, 300, 2, 8, 8, 128, 7, 40, "bf16", "f32", "token"),
    (300, 200, 1, 8, 8, 64, 5, 0, "e4m3", "f32", "token"),
    (170, 300, 1, 8, 8, 32, 1, 0, "f32", "bf16", "token"),
    (170, 300, 1, 8, 8, 64, 16, 0, "bf16", "bf16", "head"),
    (170, 300, 2, 8, 8, 128, 16, 90, "e4m3", "bf16", "head"),
    (170, 300, 1, 16, 8, 64, 48, 0, "f32", "f32", "head"),
    (140, 300, 6, 32, 8, 64, 16, 100, "bf16", "bf16", "head"),  # 24 rows
    (140, 300, 9, 24, 8, 64, 20, 60, "bf16", "f32", "token"),   # 27 rows
    (140, 300, 6, 32, 8, 128, 12, 100, "e4m3", "bf16", "token"),
]


@pytest.mark.parametrize("scale", [0.02, 0.125])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_four_heads_to_a_workgroup(case, scale):
    N, longest, m, Hq, Hkv, d, page, window, cache, out, layout = SHARED[case]
    print(f"rows {SHARED[case]} scale {scale}", flush=True)
    rng = np.random.default_rng((71, case))
    lens = [int(x) for x in rng.integers(0, longest + 1, N)]
    lens[3], lens[-1], lens[0] = 0, longest, 1
    dev, h = make((72, case), lens, m, Hq, Hkv, d, page, cache, layout)
    check(dev, h, scale, window, out)


@pytest.mark.parametrize("cache,out", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows", [(1, 4), (2, 4), (4, 5)])
def test_small_scores(cache, out, rows):
    """Weights close to each other, none of them a power of two but the largest."""
    m, G = rows
    lens = [2, 3, 40, 129, 333, 1300]
    dev, h = make((73, m, G), lens, m, 2 * G, 2, 64, 16, cache)
    check(dev, h, 0.01, 0, out)


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("N", [1, 260])
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window", [0, 45])
def test_values_that_are_not_finite_with_two_row_tiles(cache, N, page, window):
    """24 rows of six drafts. The values of the two newest tokens are not finite (NaN, then an infinity
    where the type has one), and with a window those of the two oldest: rows that see one turn
    NaN or infinite, the others stay as they are. N = 260: a wave per head; N = 1: four."""
    import torch
    m, Hq, Hkv, L, scale = 6, 32, 8, 100, 0.05
    dev, h = make((74, page), [L] * N, m, Hq, Hkv, 64, page, cache)
    bad = {L - 1: "nan", L - 2: "inf"}
    if window:  # the first draft sees L - m + 1 - window on, the last L - window on
        bad.update({L - window - 1: "nan", L - window - m + 1: "inf"})
    for tok, kind in bad.items():
        value = float(kind) if cache != "e4m3" else float("nan")
        pg = dev["block_table"][:, tok // page].long()
        x = torch.full((N, Hkv, 64), value).to(dev["v_cache"].dtype).cuda()
        dev["v_cache"].view(torch.uint8)[pg, tok % page] = x.view(torch.uint8)
        for n in range(N):
            h["v"][n][tok] = 0.0  # rows that see it are left out below
    got, _ = run(dev, scale=scale, window=window)
    o, off, _, _ = attend_rows(h["q"], h["k"], h["v"], h["lens"], scale, window, cache)
    for j in range(m):
        hi = L - m + 1 + j
        lo = max(0, hi - window) if window else 0
        sees = [kind for tok, kind in bad.items() if lo <= tok < hi]
        if not sees:
            assert not outside(got[:, j], o[:, j], off[:, j], "f32").any(), j
        elif "nan" in sees or cache == "e4m3":
            assert np.isnan(got[:, j]).all(), j
        else:
            assert np.isposinf(got[:, j]).all(), j


@pytest.mark.parametrize("cache,m", [("bf16", 1), ("e4m3", 2), ("bf16", 5)])
def test_four_heads_to_a_workgroup_captured_and_replayed(cache, m):
    """The launch that asks for more LDS than is given unasked, captured; lengths change between
    replays, with eager calls in between."""
    import torch
    from gated_delta_rule_59_amd import binding
    N, scale = 270, 0.05
    lens = [[300 - i for i in range(N)], [(7 * i) % 301 for i in range(N)], [0] * (N - 1) + [300]]
    dev, _ = make((75, m), [300] * N, m, 32, 8, 64, 16, cache, poison=False)
    want = []
    for x in lens:
        dev["seq_lens"].copy_(torch.tensor(x))
        want.append(binding.paged_decode(**dev, scale=scale))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = binding.paged_decode(**dev, scale=scale)
    for i in (0, 1, 2, 1, 0):
        dev["seq_lens"].copy_(torch.tensor(lens[i]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i])
        assert torch.equal(binding.paged_decode(**dev, scale=scale), want[i])
        torch.cuda.synchronize()
    assert (want[2][:-1] == 0).all() and (want[2][-1] != 0).any()
