"""dsa_beam_select where totals are equal: signed zeros, beams that are the
same; and the sums of long rows of equal logits."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_beam import DT, D, rand, run  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("zeros", [40, 180, 700, 39000])
def test_zeros_of_either_sign_are_equal(D, dtype, zeros):  # noqa: F811
    """Lists that are handed on as they are, ranked, and cut: -0 at lower tokens, +0 at higher ones."""
    V = 40001
    x = torch.full((2, V), -3.0, device="cuda")
    at = torch.linspace(0, V - 1, zeros, device="cuda").long()
    x[:, at] = 0.0
    x[0, at[:zeros // 2]] = -0.0
    x[1, at[::2]] = -0.0
    run(D, x.to(DT[dtype]), torch.tensor([0.0, -1.0], device="cuda"), 1, 2, 16)


def test_zero_scores_of_either_sign_are_equal(D):  # noqa: F811
    x, _ = rand(4, 999, "fp32", 2)
    done = torch.ones(4, dtype=torch.uint8, device="cuda")
    for s in ([-0.0, 0.0, 0.0, -0.0], [0.0, -0.0, -0.0, 0.0]):
        for select in (1, 2, 3):
            run(D, x, torch.tensor(s, device="cuda"), 1, 4, select, finished=done, pad=7)
            run(D, x, torch.tensor(s, device="cuda"), 2, 2, select, finished=done, pad=7)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("batch,beams,V,select", [(1, 4, 131072, 8), (3, 5, 50001, 10), (1, 64, 30011, 64), (9, 8, 131073, 16),
                                                  (40, 4, 9001, 4), (1, 2, 260000, 2)])
def test_beams_that_are_the_same_tie(D, dtype, batch, beams, V, select):  # noqa: F811
    """Beams of the same logits and score, though cut into other slices and aligned otherwise: their totals
    are equal, so the lower one's come first. Beside them others of another score, or nearly the same row."""
    x, s = rand(batch * beams, V, dtype, V + beams)
    for b in range(batch):
        rows = x[b * beams:(b + 1) * beams]
        rows[:] = rows[0].clone()
        s[b * beams:(b + 1) * beams] = s[b * beams].clone()
        if beams >= 4:
            s[b * beams + 1] -= 0.125          # another score (exact in fp32, as its multiples)
            rows[3, V // 2] = -math.inf        # another row
    run(D, x, s, batch, beams, select)
    # the first step as it is often written: every beam but the first far behind, all rows alike
    x = x[:beams].clone()
    x[:] = x[0].clone()
    s = torch.full((beams,), -1e9, device="cuda")
    s[0] = 0
    run(D, x, s, 1, beams, min(64, select + 2))


@pytest.mark.parametrize("dtype,value", [("bf16", 0.30078125), ("fp16", -4.19921875), ("fp32", 0.1), ("fp32", -7.3)])
@pytest.mark.parametrize("rows,V", [(500, 1 << 17), (460, (1 << 20) + 3)])
def test_sums_of_long_rows_of_equal_logits(D, dtype, value, rows, V):  # noqa: F811
    """log sum exp is x + log V. Every addition in a row of equal terms rounds the same way: the sums must not
    let that grow with the row (they are good to 1e-6, and the score is rounded to fp32)."""
    x = torch.full((rows, V), value, device="cuda", dtype=DT[dtype])
    s = torch.zeros(rows, device="cuda")
    p = D.make_beam_problem(rows, 1, V, 2, dtype)
    outs = (torch.empty(rows, 2, device="cuda"), torch.empty(rows, 2, dtype=torch.int32, device="cuda"),
            torch.empty(rows, 2, dtype=torch.int32, device="cuda"))
    D.dsa_beam_select(p, x, s, *outs, D.alloc_beam_workspace(p))
    got = outs[0].double().cpu().numpy()
    want = -math.log(V)
    assert (np.abs(got - want) <= 1e-6 + abs(want) * 2.0 ** -24).all(), np.abs(got - want).max()
    assert (outs[1].cpu().numpy() == [0, 1]).all()
