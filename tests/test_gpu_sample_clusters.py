"""dsa_sample's ways through the kernel, side by side in rows of one call whose blocks form clusters: empty
rows, the largest logit alone, ties beyond a list, lists, cuts in one bin and in several. Every call gives the
same bits."""
import math

import pytest
import torch

from tests.test_gpu_sample import D, logits_of, reference, uniform  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,dtype", [(2, 131072, "bf16"), (12, 131072, "bf16"), (18, 100001, "fp16"), (12, 300000, "fp32"), (36, 60000, "bf16")])
def test_rows_that_leave_in_every_way(D, rows, vocab, dtype):  # noqa: F811
    x = logits_of(rows, vocab, dtype, seed=rows)
    heat, k, p, low = torch.ones(rows), torch.zeros(rows, dtype=torch.int32), torch.ones(rows), torch.zeros(rows)
    for r in range(rows):
        way = (r + vocab) % 9
        if way == 0:
            x[r] = -math.inf
        elif way == 1:
            heat[r] = 0.0
        elif way == 2:
            x[r, vocab // 2:] = math.inf                        # more of the largest than a list holds
        elif way == 3:
            k[r] = 30
        elif way == 4:
            k[r], p[r] = 5000, 0.9
        elif way == 5:
            p[r] = 0.95
        elif way == 6:
            x[r], p[r] = 1.0, 0.3                               # one value
        elif way == 7:
            low[r] = 0.01
    u = uniform(rows, 3)
    dev = [t.cuda() for t in (x, u, heat, k, p, low)]
    plan = D.make_sample_problem(rows, vocab, dtype)
    n = 60
    tok, lp = torch.full((n, rows), -9, dtype=torch.int32, device="cuda"), torch.full((n, rows), 9.0, device="cuda")
    for i in range(n):
        D.dsa_sample(plan, dev[0], dev[1], tok[i], temperature=dev[2], top_k=dev[3], top_p=dev[4], min_p=dev[5], logprobs=lp[i])
    assert (tok == tok[0]).all() and (lp.view(torch.int32) == lp[0].view(torch.int32)).all()
    for r in range(rows):
        want, wlp, near = reference(x[r].double().numpy(), float(u[r]), float(heat[r]), int(k[r]), float(p[r]), float(low[r]))
        if near < 2.0 ** -29:
            continue
        got = float(lp[0, r])
        assert int(tok[0, r]) == want and (got == wlp or abs(got - wlp) <= 2.0 ** -29 + abs(wlp) * 2.0 ** -21), r
