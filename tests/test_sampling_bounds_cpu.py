"""The sampler's fp32 steps from a logit to the grid point of its weight's logarithm, restated here: what lies
beyond the point stays within the bound that the bins' bounds are made with, and a token's distance below its
bin's edge is never counted as less than zero."""
import os
import re

import numpy as np
import pytest

import top_sparse_attention_chunked_gb300 as pkg

F = np.float32


def constant(name):
    with open(os.path.join(os.path.dirname(pkg.__file__), "csrc", "sample.cu")) as f:
        m = re.search(rf"\b{name} = ([0-9.]+)f?;", f.read())
    assert m, f"{name} is not in the source"
    return float(m.group(1))


def residual(x, heat):
    """Points (512 to a factor of two) that x's exponent has beyond its grid point, for logits below 4,096 in log2 units."""
    c = 1.4426950408889634 / float(F(heat))
    ch = F(c)
    cl = F(c - float(ch))
    d = x.astype(np.float64)
    n = F(d * float(ch))                                   # (48 bits: the product is exact in 64)
    t = F(n.astype(np.float64) + 24576.0)                  # adding 1.5 * 2^14 rounds to multiples of 1 / 512
    k = F(t.astype(np.float64) - 24576.0)
    inner = F(d * float(ch) - n.astype(np.float64))
    r = F(F(n - k).astype(np.float64) + F(d * float(cl) + inner.astype(np.float64)).astype(np.float64))
    return r.astype(np.float64) * 512


@pytest.mark.parametrize("heat", [0.005, 0.01, 0.033, 0.72, 1.0, 1.7, 9.3, 250.0])
def test_distances_are_positive_and_within_the_bound(heat):
    rng = np.random.default_rng(int(heat * 1000))
    most = 4096 * float(F(heat)) / 1.4426950408889634
    x = F(np.concatenate([rng.uniform(most * 0.5, most, 500000), rng.uniform(-most, most, 200000),
                          -rng.uniform(most, most * (1 + 80 / 4096), 300000)]))     # (what is below the largest: 80 further)
    r = residual(x, heat)
    assert np.abs(r).max() > 0.55, "no logit comes near the bound"
    assert np.abs(r).max() <= constant("kRest")
    under = constant("kBelow") + np.rint(-r * 64)          # of a token at its bin's edge
    assert under.min() >= 0
