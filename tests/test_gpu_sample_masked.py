"""dsa_sample on rows of which whole stretches are masked, as in constrained decoding or a vocabulary padded at
its end: the token of 64 bits, and no slower than the rows without a mask."""
import math

import pytest
import torch

from tests.test_gpu_sample import D, logits_of, run, uniform  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu

SETTINGS = [dict(k=50), dict(k=50, p=0.9), dict(k=600, heat=1.5), dict(p=0.9), dict(p=0.3, heat=0.7), dict(k=3000, p=0.99), dict(heat=0.0), dict(low=0.1), dict()]


def masks(vocab):
    """Which tokens stay."""
    at = torch.arange(vocab)
    g = torch.Generator().manual_seed(vocab)
    some = torch.zeros(vocab, dtype=torch.bool)
    some[torch.randperm(vocab, generator=g)[:300]] = True
    return [at < vocab * 7 // 8, at >= vocab // 2, (at * 8 // vocab) % 2 == 1, at < 40, (at > vocab // 3) & (at < vocab // 3 + 500), some,
            (at * 8 // vocab == 3) | (at == 5), at == vocab - 1]


@pytest.mark.parametrize("vocab,dtype", [(131072, "bf16"), (50257, "fp16"), (200003, "fp32")])
def test_masked_stretches(D, vocab, dtype):  # noqa: F811
    keep = torch.stack(masks(vocab))
    for least in (-math.inf, torch.finfo(torch.float16 if dtype == "fp16" else torch.float32).min):
        x = logits_of(len(keep), vocab, dtype, seed=3)
        x = torch.where(keep, x, torch.tensor(least, dtype=x.dtype))
        for i, s in enumerate(SETTINGS):
            run(D, x, uniform(len(keep), i), **s)


def test_rows_of_lists_that_overflow(D):  # noqa: F811
    """More finite tokens than a list holds, fewer threads' worth than it asks for."""
    for vocab in (1025, 1500, 2039, 2050):
        x = logits_of(6, vocab, "bf16", seed=vocab)
        for i, s in enumerate(SETTINGS):
            run(D, x, uniform(6, i), **s)


def timed(D, x, k, p):  # noqa: F811
    n = x.shape[0]
    f = lambda v, t: None if v is None else torch.full((n,), v, dtype=t, device="cuda")  # noqa: E731
    plan, u, tok = D.make_sample_problem(n, x.shape[1], "bf16"), f(0.37, torch.float32), f(0, torch.int32)
    kk, pp = f(k, torch.int32), f(p, torch.float32)
    D.dsa_sample(plan, x, u, tok, top_k=kk, top_p=pp)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(20):
            D.dsa_sample(plan, x, u, tok, top_k=kk, top_p=pp)
    best = math.inf
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / 20)
    return best


@pytest.mark.parametrize("rows", [1, 64])
@pytest.mark.parametrize("k,p", [(50, None), (50, 0.9)])
def test_a_mask_costs_no_further_passes(D, rows, k, p):  # noqa: F811
    """Half of every row masked: 1.7 to 2.9 times as long where every token was offered to the list."""
    x = logits_of(rows, 131072, "bf16", std=1.6, seed=rows, peaks=40).cuda()
    y = x.clone()
    y[:, 65536:] = -math.inf
    whole, half = timed(D, x, k, p), timed(D, y, k, p)
    assert half <= 1.4 * whole, f"{half * 1e3:.1f} us with a mask, {whole * 1e3:.1f} without"
