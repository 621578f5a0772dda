"""dsa_rope_axes_append with positions that are a slice of a longer buffer, or one row for all axes."""
import pytest
import torch

from tests.test_gpu_rope_axes import D, make  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu


def call(D, c, pos, in_turn):  # noqa: F811
    q, k, v = c["qkv"].cuda().split(c["split"], 1)
    p = D.make_rope_axes_problem(c["tokens"], c["hq"], c["hkv"], c["rows"], c["sections"], c["max_pos"], in_turn)
    out = torch.zeros(c["tokens"], c["hq"], 128, device="cuda", dtype=torch.bfloat16)
    K, V = (torch.zeros(c["rows"], c["hkv"], 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    D.dsa_rope_axes_append(p, q, k, v, *(c[n].cuda() for n in ("gq", "gk", "cos", "sin")), pos, c["slots"].cuda(), out, K, V)
    return out, K, V


@pytest.mark.parametrize("tokens", [1, 5, 130])
@pytest.mark.parametrize("sections", [(16, 24, 24), (20, 13), (64,)])
def test_slices_of_a_longer_buffer(D, tokens, sections):  # noqa: F811
    c = make(tokens, 6, 2, sections, seed=tokens)
    long = torch.full((len(sections), 700), 10 ** 9, dtype=torch.int32, device="cuda")
    for off in (0, 3):
        view = long[:, off:off + tokens]
        view.copy_(c["pos"])
        for in_turn in (False, True):
            for a, b in zip(call(D, c, c["pos"].cuda(), in_turn), call(D, c, view, in_turn)):
                assert torch.equal(a, b)
    same = c["pos"][:1].cuda()
    for a, b in zip(call(D, c, same.repeat(len(sections), 1), False), call(D, c, same.expand(len(sections), tokens), False)):
        assert torch.equal(a, b)
