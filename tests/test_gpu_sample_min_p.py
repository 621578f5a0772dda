"""dsa_sample's min-p cut to the last bit of the logits.

A row's logits rise from below the cut, max + T ln min_p, to above it, an fp32 step apart, so that a random
number of 0 takes the first that is kept. Where max and T ln min_p nearly cancel, a step of the logits is far
less than a step of either."""
import math
import random

import pytest
import torch

from tests.test_gpu_sample import D  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu

AROUND = 40


def rows_of(seed, n, cancel):
    """(logits [n, 2 AROUND + 2], temperature, min_p, the first kept) with the cut in 64 bits."""
    r = random.Random(seed)
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    x, heat, low, want = [], [], [], []
    while len(x) < n:
        t, p = f32(r.choice([1.0, 0.7, 2.5, 0.05, 13.0, r.uniform(0.1, 3)])), f32(10 ** r.uniform(-6, -0.01))
        d = t * math.log(p)                                      # (right to 2^-50 of itself)
        top = f32(-d * (1 + 10 ** r.uniform(-6, -1)) if cancel else r.choice([0.0, r.uniform(-30, 30), r.uniform(-2000, 2000)]))
        cut = top + d
        mid = torch.tensor(cut, dtype=torch.float32)
        if mid.abs() < 1e-30 or float(mid) >= top:
            continue
        near = [mid]
        for _ in range(AROUND):
            near.insert(0, torch.nextafter(near[0], torch.tensor(-math.inf)))
            near.append(torch.nextafter(near[-1], torch.tensor(math.inf)))
        row = [float(v) for v in near]
        # (the cut is known to 2^-49 of max and T ln min_p: no logit is nearer than 16 times that)
        if row[-1] >= top or min(abs(v - cut) for v in row) < 2.0 ** -45 * (abs(top) + abs(d)):
            continue
        x.append(row + [top])
        heat.append(t)
        low.append(p)
        want.append(next(i for i, v in enumerate(row) if v > cut))
    return torch.tensor(x), torch.tensor(heat), torch.tensor(low), want


@pytest.mark.parametrize("cancel", [True, False])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_cut_to_the_last_bit(D, cancel, seed):  # noqa: F811
    n = 500
    x, heat, low, want = rows_of(seed, n, cancel)
    tok = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    plan = D.make_sample_problem(n, x.shape[1], "fp32")
    D.dsa_sample(plan, x.cuda(), torch.zeros(n, device="cuda"), tok, temperature=heat.cuda(), min_p=low.cuda())
    wrong = [(i, t, w) for i, (t, w) in enumerate(zip(tok.tolist(), want)) if t != w]
    assert not wrong, f"{len(wrong)} of {n} rows, the first {wrong[:5]}"


def test_cutoffs_that_leave_the_range(D):  # noqa: F811
    """min_p of 1, above 1 and next to 0, temperatures whose product with ln min_p is infinite, logits at the type's ends."""
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[-1.0, 0.5, 2.0, 1.999999]] * 6 + [[-big, 0.0, big, -1.0]] * 3)
    heat = torch.tensor([1.0, 1.0, 1.0, math.inf, 3e38, 1e-30, 1.0, math.inf, 3e38])
    low = torch.tensor([1.0, 7.0, 1e-38, 0.5, 1e-38, 0.5, 0.5, 0.5, 0.01])
    tok = torch.full((9,), -9, dtype=torch.int32, device="cuda")
    D.dsa_sample(D.make_sample_problem(9, 4, "fp32"), x.cuda(), torch.zeros(9, device="cuda"), tok, temperature=heat.cuda(), min_p=low.cuda())
    assert tok.tolist() == [2, 2, 0, 0, 0, 2, 2, 0, 0]
