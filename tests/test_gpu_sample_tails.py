"""dsa_sample with a nucleus that ends among tokens of less than 2^-32 of the largest's weight.

One heavy token, thousands that share a value some 2^-32 of it, and the cut a little beyond them, among the
tokens of a third value. These come first in the row, so that a random number of 0 takes the first of them if
the cut is where it belongs, and another token if it is not. Weights are right to 2^-45 of the largest each:
the cut lies further from every border than all of that together."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_sample import D, DT, run, uniform  # noqa: F401 (D is a fixture)
from tests.test_sampling_bounds_cpu import residual

pytestmark = pytest.mark.gpu

# type, temperature, the heavy logit, the shared one and how many have it, the third one and how many
ROWS = [("fp16", 0.7, -16.40625, -31.921875, 130521, -32.0625, 9974), ("fp16", 0.7, -16.40625, -31.921875, 74577, -32.90625, 8963),
        ("bf16", 5.0, 104.0, -6.90625, 25325, -13.8125, 6879), ("bf16", 0.7, 0.020751953125, -15.5, 45644, -16.0, 3453),
        ("fp16", 5.0, 55.53125, -55.375, 24179, -56.40625, 1505), ("fp16", 5.0, 0.159912109375, -110.6875, 124067, -111.75, 1294),
        ("bf16", 0.7, 0.025146484375, -15.5, 62799, -16.0, 2926), ("fp32", 1.0, 0.0, -22.1765, 70000, -22.5, 3000)]


@pytest.mark.parametrize("dtype,heat,top,shared,many,third,few", ROWS)
def test_cut_below_the_last_bin(D, dtype, heat, top, shared, many, third, few):  # noqa: F811
    p = 1 - 2.0 ** -24
    x = torch.full((1, 1 + many + few), shared)
    x[0, :few] = third
    x[0, few] = top
    x = x.to(DT[dtype])
    # the running sums' borders, in 64 bits, and the documented error of all weights
    heat32 = float(torch.tensor(heat))
    v = [float(x[0, i].double()) for i in (few, few + 1, 0)]
    w1, w2 = (math.exp((a - v[0]) / heat32) for a in v[1:])
    total = math.fsum([1.0, many * w1, few * w2])
    last = (p * total - 1 - many * w1) / w2            # of the third value's tokens
    error = (1 + many + few) * 2.0 ** -45 + total * 2.0 ** -31
    assert error < last * w2 and error < (few - last) * w2, "the cut is next to a border"
    tok, lp = torch.full((1,), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    plan = D.make_sample_problem(1, x.shape[1], dtype)
    f = lambda t: torch.tensor([t], dtype=torch.float32, device="cuda")  # noqa: E731
    for k in (None, 1 + many + few - 1):
        ks = None if k is None else torch.tensor([k], dtype=torch.int32, device="cuda")
        D.dsa_sample(plan, x.cuda(), f(0.0), tok, temperature=f(heat), top_k=ks, top_p=f(p), logprobs=lp)
        assert int(tok) == 0, f"the third value's first token is kept, token {int(tok)} came"
        want = math.log(w2 / (1 + many * w1 + math.ceil(last) * w2))
        assert abs(float(lp) - want) <= 2.0 ** -20 * abs(want) + 2.0 ** -28


@pytest.mark.parametrize("heat", [0.005, 0.01, 0.72])
def test_heavy_logit_far_beyond_its_grid_point(D, heat):  # noqa: F811
    """The largest logit alone in its bin, and above the bin's edge by as much as fp32 steps leave it."""
    most = 4096 * heat / 1.4426950408889634
    x0 = np.random.default_rng(5).uniform(most * 0.5, most, 300000).astype(np.float32)
    r = residual(x0, heat)
    tops = torch.from_numpy(x0[np.argsort(-r)[:6]].copy())
    assert r.max() > 0.626
    g = torch.Generator().manual_seed(9)
    z = (torch.randn(6, 60000, generator=g) * 0.8).clamp(max=3)
    x = tops[:, None] + (z - 6) * heat
    x[:, 777] = tops
    for i, s in enumerate((dict(p=0.9), dict(p=0.3), dict(p=torch.linspace(0.02, 0.999, 6)), dict(k=20000, p=0.7), dict(k=50, p=0.9))):
        run(D, x, uniform(6, i), heat=heat, **s)
