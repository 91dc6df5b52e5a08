"""How many bits prompts of linear attention hold: keys and queries of one channel each, so that a result is a
sum of few terms and nothing hides what a term is off by.

In units of u = 2^-24 of a term: e^x is off by 4 (the instruction's 2, its exponent's rest 1, their product 1).
One chunk. S: e^x 4, times the value 1, three bf16 parts and their sums 2.5 (fp32: one product, 1), the
state's own factor 5, the sum with S0 1: 14. o: e^x 4, the scale 1, times q k 1, the parts 2.5, the sum with
the state's term 3 (which has e^x 4, scale 1, product 1, parts 2.5): 14. A state of two bf16 parts would be off by 64,
an exponent rounded to 32 bits by 11 for decays of 2^-16 to 2^-32.
Several chunks and segments: S once more the factor of each of the two segments before (5 each, and the sum 1),
the segment's own sum (5), a sum per token of a channel (3): 34. o: those and its own 14: 48.
Then o's rounding: half a step."""
import numpy as np
import pytest

from tests.step_ref import lin
from tests.test_gpu_lin import dev, rounded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")]


def one_channel_each(seed, T, H, dk, dv, n_seq, act, powers):
    """Token t's key is channel t % dk, its query any; a sequence decays by 2^-powers, unevenly."""
    rng = np.random.default_rng(seed)
    q, k = np.zeros((T * n_seq, 1, dk)), np.zeros((T * n_seq, 1, dk))
    t = np.arange(T * n_seq)
    q[t, 0, rng.integers(0, dk, T * n_seq)] = rng.standard_normal(T * n_seq)
    k[t, 0, t % T % dk] = rng.standard_normal(T * n_seq)
    v = rng.standard_normal((T * n_seq, H, dv))
    g = rng.random((n_seq, T, H)) ** 2 + 1e-3
    g = -powers * np.log(2.0) * g / g.sum(1, keepdims=True)
    S0 = rng.standard_normal((n_seq, H, dk, dv)).astype(np.float32)
    return (*(rounded(x, act) for x in (q, k, v)), rounded(g.reshape(T * n_seq, H), "f32"), S0)


def half_step(want, out):
    """Half of what the result's type steps by at `want`."""
    e = np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -120)))
    return 2.0 ** (e - (8 if out == "bf16" else 24))


def check(x, B, act, out, units_o, units_S, scale=0.3):
    import torch
    from gated_delta_rule_59_amd import binding
    q, k, v, g, S0 = x
    T = q.shape[0] // B
    view = lambda t: t.view(B, T, *t.shape[1:])  # noqa: E731
    scale = float(np.float32(scale))
    o, S = binding.lin_chunk_fwd(view(dev(q, act)), view(dev(k, act)), view(dev(v, act)), view(dev(g)), dev(S0),
                                 scale=scale, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    torch.cuda.synchronize()
    ro, rS, ao, A = lin(q, k, v, g, S0, scale, [T] * B)
    err = np.abs(o.double().cpu().numpy().reshape(ro.shape) - ro) - half_step(ro, out)
    worst = (err / (U * ao + 1e-35)).max()
    assert worst <= units_o, f"o: {worst:.1f} units"
    worst = (np.abs(S.double().cpu().numpy() - rS) / (U * A + 1e-35)).max()
    assert worst <= units_S, f"S: {worst:.1f} units"


@pytest.mark.parametrize("powers", [0.5, 10, 23.5, 31, 60])
@pytest.mark.parametrize("act,out", TYPES)
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128), (128, 32), (64, 64)])
def test_one_chunk(dk, dv, act, out, powers):
    T = 64 if act == "bf16" else 32
    print(f"lin one chunk {dk}x{dv} {act} {out} 2^-{powers}", flush=True)
    check(one_channel_each((31, dk, dv, int(2 * powers)), T, 4, dk, dv, 6, act, powers), 6, act, out, 14, 14)


@pytest.mark.parametrize("powers", [0.5, 10, 23.5])
@pytest.mark.parametrize("act,out", TYPES)
def test_segments(act, out, powers):
    print(f"lin segments {act} {out} 2^-{powers}", flush=True)
    check(one_channel_each((32, int(2 * powers)), 384, 3, 128, 64, 1, act, powers), 1, act, out, 48, 34)
